"""The 8-bit outputs are what their definition gives in fp32, bit for bit: scale = largest magnitude times the fp32 number
next to 1/448 (at least 2^-126), value = the quotient by that scale rounded to nearest, then e4m3 rounded to nearest
even. (The norm's outputs in 8 bits are held to its own fp32 output, which is what they are made of.)"""
import pytest
import torch

from ag_gemm_gb300 import binding as B

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need a GB300"
    return torch.device("cuda:0")


def in_8_bits(x, up):
    """x [rows, cols] fp32 on the CPU -> its e4m3 bytes and scales, by IEEE arithmetic."""
    rows, cols = x.shape
    a, b = -(-rows // up), -(-cols // 128)
    p = torch.zeros(a * up, b * 128)
    p[:rows, :cols] = x
    p = p.view(a, up, b, 128)
    scale = torch.maximum(p.abs().amax(dim=(1, 3)) * torch.tensor(1.0 / 448.0), torch.tensor(2.0 ** -126))
    q = (p / scale[:, None, :, None]).clamp(-448, 448).to(E4M3)
    return q.view(torch.uint8).reshape(a * up, b * 128)[:rows, :cols], scale


def near_borders(g, rows, cols, up):
    """Values that lie on the borders between two 8-bit numbers, and a few fp32 steps beside them, under scales of any
    size (those too that are not powers of two)."""
    a, b = -(-rows // up), -(-cols // 128)
    exps = 12 if up == 1 else 6
    scale = torch.exp2(torch.randint(-exps, exps, (a, b), generator=g).float()) * (1 + torch.randint(0, 16, (a, b), generator=g) / 16)
    each = scale.repeat_interleave(up, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    border = (torch.randint(8, 16, (rows, cols), generator=g) + 0.5) * torch.exp2(torch.randint(-9, 6, (rows, cols), generator=g).float())
    v = border * each * torch.where(torch.rand(rows, cols, generator=g) < 0.5, -1.0, 1.0)
    v = v * (1 + torch.randint(-2, 3, (rows, cols), generator=g) * 2.0 ** -23)
    v = v.clamp(-448, 448).minimum(448 * each).maximum(-448 * each)
    v[::up, ::128] = 448 * scale                      # the scale's own value
    return v


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["borders", "normal", "small", "large"])
@pytest.mark.parametrize("rows,cols", [(256, 1024), (300, 1040), (131, 1357), (64, 258), (300, 132)])
@pytest.mark.parametrize("up", [1, 128])
def test_quantised_values_are_the_definitions(dev, up, rows, cols, kind, dtype):
    g = torch.Generator().manual_seed(rows + cols + up)
    if kind == "borders":
        x = near_borders(g, rows, cols, up)
    else:
        x = torch.randn(rows, cols, generator=g) * {"normal": 1.0, "small": 1e-36, "large": 1e37}[kind]
    x = x.to(TYPES[dtype])
    want, scales = in_8_bits(x.float(), up)
    a, b = scales.shape
    q, scale = torch.empty(rows, cols, dtype=torch.uint8, device=dev), torch.empty(a, b, device=dev)
    copy = dict(qt=[torch.empty(cols, rows, dtype=torch.uint8, device=dev)], scale_t=[torch.empty(b, a, device=dev)]) if up == 128 else {}
    B.fo_quant_fp8(rows, cols, [x.to(dev)], [q], [scale], block_rows=up, **copy)
    assert torch.equal(scale.cpu(), scales)
    assert torch.equal(q.cpu(), want)
    if copy:
        assert torch.equal(copy["qt"][0].cpu(), want.t())


@pytest.mark.parametrize("cols", [384, 388, 387])
@pytest.mark.parametrize("up", [1, 128])
def test_special_values_in_bf16(dev, up, cols):
    """Infinities, NaN of either sign and zeros of either sign in bf16, whose magnitudes are compared as they are read."""
    x = torch.randn(256, cols, generator=torch.Generator().manual_seed(cols)).bfloat16()
    x[3, 7] = -50.0                                    # the largest magnitude is a negative value's
    x[5, ::2] = -0.0
    x[130, 5] = float("-inf")
    x[200, 300] = float("nan")
    x.view(torch.int16)[201, 130] = -1                 # a negative NaN, the largest of them
    want, scales = in_8_bits(x.float(), up)
    q, scale = torch.empty(256, cols, dtype=torch.uint8, device=dev), torch.empty(scales.shape, device=dev)
    B.fo_quant_fp8(256, cols, [x.to(dev)], [q], [scale], block_rows=up)
    q, scale = q.cpu(), scale.cpu()
    assert torch.equal(torch.isnan(scale), torch.isnan(scales)) and torch.isnan(scale).sum() == 2
    assert torch.equal(scale.nan_to_num(nan=1.0), scales.nan_to_num(nan=1.0)) and torch.isinf(scale).sum() == 1
    nan, nans = torch.isnan(q.view(E4M3).float()), torch.isnan(want.view(E4M3).float())
    assert torch.equal(nan, nans) and nan[130, 5] and nan[200, 300] and nan[201, 130]
    assert torch.equal(q[~nan], want[~nan])


@pytest.mark.parametrize("rows,H", [(700, 4096), (300, 1024), (50, 1357), (20, 16384), (9, 32768), (400, 260)])
def test_norms_8_bits_are_those_of_its_output(dev, rows, H):
    g = torch.Generator().manual_seed(rows + H)
    x, w = torch.randn(rows, H, generator=g).to(dev), (1 + 0.2 * torch.randn(H, generator=g)).to(dev)
    y, q, scale = torch.empty_like(x), torch.empty(rows, H, dtype=torch.uint8, device=dev), torch.empty(rows, -(-H // 128), device=dev)
    B.fo_rmsnorm(B.fo_norm_desc(H, dtype="f32"), rows, [x], None, w, None, [y], [q], [scale])
    want, scales = in_8_bits(y.cpu(), 1)
    assert torch.equal(scale.cpu(), scales)
    assert torch.equal(q.cpu(), want)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,H", [(700, 4096), (300, 1024), (50, 1358), (90, 1357), (20, 16384), (400, 260)])
def test_norms_8_bits_in_bf16_are_those_of_its_formula(dev, rows, H, residual):
    """From its own rstd on, the norm's outputs are its formula's in fp32, operation by operation."""
    g = torch.Generator().manual_seed(rows + H)
    x, res = (torch.randn(rows, H, generator=g).bfloat16() for _ in range(2))
    w = (1 + 0.2 * torch.randn(H, generator=g)).bfloat16()
    y, q = torch.empty(rows, H, dtype=torch.bfloat16, device=dev), torch.empty(rows, H, dtype=torch.uint8, device=dev)
    scale, rstd = torch.empty(rows, -(-H // 128), device=dev), torch.empty(rows, device=dev)
    B.fo_rmsnorm(B.fo_norm_desc(H), rows, [x.to(dev)], [res.to(dev)] if residual else None, w.to(dev), None, [y], [q], [scale], [rstd])
    s = x.float() + res.float() if residual else x.float()
    n = s * rstd.cpu()[:, None] * w.float()
    want, scales = in_8_bits(n, 1)
    assert torch.equal(scale.cpu(), scales) and torch.equal(q.cpu(), want) and torch.equal(y.cpu(), n.bfloat16())
