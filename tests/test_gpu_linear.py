"""Projections with group-quantized weights against the 64-bit sum (block_ref.linear states the bound)."""
import numpy as np
import pytest

import block_ref as ref
from helpers import bf16_tensor, bf16_to_np_bits
from workloads import gen

pytestmark = pytest.mark.gpu


def make(N, K, bits, group, seed=0):
    rng = np.random.default_rng([seed, N, K, bits, group])
    if bits == 4:
        codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)          # every nibble, -8 among them
    else:
        codes = rng.integers(0, 256, (N, K), dtype=np.uint8)               # every byte, -128 among them
    scales = (rng.uniform(0.5, 1.5, (N, K // group)) * 0.06 / (7 if bits == 4 else 127)).astype(np.float16)
    return codes, scales


def acts(T, K, seed=0):
    return gen.f32_to_bf16_bits(np.random.default_rng([seed, T, K]).standard_normal((T, K), dtype=np.float32))


def run(x_bits, codes, scales, bits, group, bias=None, residual=None, x_pad=0, out_pad=0, in_place=False):
    import torch
    import int4_grouped_expert_gb300 as st
    T, K = x_bits.shape
    N = codes.shape[0]
    wide = np.full((T, K + x_pad), 0x7FC0, dtype=np.uint16)                # nan between the rows
    wide[:, :K] = x_bits
    x = bf16_tensor(wide)
    lin = st.QuantLinear(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), N, K, bits, group,
                         bias=None if bias is None else torch.from_numpy(bias).cuda())
    out = torch.full((T + 1, N + out_pad), -7.0, dtype=torch.bfloat16, device="cuda")
    res = None
    if residual is not None:
        res = bf16_tensor(residual)
        if in_place:
            out[:T, :N] = res
            res = out
    need = lin.workspace_size(T)
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")       # no initialisation needed
    st.check(st.strata_linear_forward(lin.struct(), x, T, out, ws, need, x_stride=K + x_pad, residual=res,
                                      residual_stride=N + out_pad if in_place else N,
                                      out_stride=N + out_pad), "strata_linear_forward")
    torch.cuda.synchronize()
    o = out.cpu().float().numpy()
    assert (o[T] == -7).all() and (o[:T, N:] == -7).all(), "written outside the output rows"
    return ref.bf16_bits_to_f64(bf16_to_np_bits(out[:T, :N].contiguous()))


def check(T, N, K, bits, group, with_bias=False, with_res=False, **kw):
    import int4_grouped_expert_gb300 as st
    codes, scales = make(N, K, bits, group)
    x = acts(T, K)
    rng = np.random.default_rng(3)
    bias = rng.standard_normal(N).astype(np.float32) if with_bias else None
    res = gen.f32_to_bf16_bits(rng.standard_normal((T, N), dtype=np.float32)) if with_res else None
    got = run(x, codes, scales, bits, group, bias, res, **kw)
    want, bound = ref.linear(ref.bf16_bits_to_f64(x), codes, scales, bits, group, bias,
                             None if res is None else ref.bf16_bits_to_f64(res),
                             rounded_weights=T > st.LINEAR_EXACT_T)
    worst = (np.abs(got - want) / bound).max()
    print(f"T {T} N {N} K {K} w{bits} g{group}: worst error / bound {worst:.3f}")
    assert worst <= 1


@pytest.mark.parametrize("bits,group", [(4, 64), (4, 128), (4, 256), (8, 64), (8, 128), (8, 256)])
@pytest.mark.parametrize("T", [1, 7, 8, 9, 16, 17, 32, 33, 64, 65, 200, 257])
def test_every_format_and_batch(T, bits, group):
    check(T, 145, 768, bits, group)


@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 127, 128, 129, 1000])
@pytest.mark.parametrize("T", [3, 70])
def test_odd_widths(T, N):
    check(T, N, 512, 4, 128)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("K,group", [(64, 64), (192, 64), (128, 128), (384, 128), (1152, 128), (256, 256),
                                     (768, 256), (7168, 128)])
@pytest.mark.parametrize("T", [1, 20, 90])
def test_contraction_lengths(T, K, group, bits):
    check(T, 80, K, bits, group)


@pytest.mark.parametrize("T", [1, 12, 40, 300])
def test_bias_residual_and_strides(T):
    check(T, 515, 1024, 4, 128, with_bias=True)
    check(T, 515, 1024, 8, 64, with_res=True)
    check(T, 515, 1024, 4, 64, with_bias=True, with_res=True, x_pad=8, out_pad=3)
    check(T, 512, 1024, 8, 128, with_bias=True, with_res=True, x_pad=40, out_pad=1, in_place=True)


@pytest.mark.parametrize("bits", [4, 8])
def test_a_wide_layer(bits):
    check(16, 6145, 4096, bits, 128)
    check(129, 6145, 4096, bits, 128)


@pytest.mark.parametrize("T", [5, 96])
def test_large_and_small_activations(T):
    """Rows far outside the f16 range on either side keep their relative precision."""
    codes, scales = make(64, 512, 4, 128)
    x = ref.bf16_bits_to_f64(acts(T, 512))
    x *= np.exp2(np.linspace(-40, 40, T).round())[:, None]
    bits = gen.f32_to_bf16_bits(x.astype(np.float32))
    got = run(bits, codes, scales, 4, 128)
    want, bound = ref.linear(ref.bf16_bits_to_f64(bits), codes, scales, 4, 128, rounded_weights=T > 32)
    assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("T", [6, 50])
def test_non_finite_rows_stay_alone(T):
    codes, scales = make(100, 512, 8, 128)
    scales[37, 2] = np.nan                                                # a group that held inf or nan
    x = acts(T, 512)
    x[2, 11], x[4, 100] = 0x7FC0, 0x7F80                                  # a nan and an inf
    got = run(x, codes, scales, 8, 128)
    rows, cols = np.arange(T) != 2, np.arange(100) != 37
    assert np.isnan(got[2]).all() and np.isnan(got[:, 37]).all()
    rows[4] = False
    want, bound = ref.linear(ref.bf16_bits_to_f64(x[rows]), codes[cols], scales[cols], 8, 128,
                             rounded_weights=T > 32)
    assert (np.abs(got[rows][:, cols] - want) <= bound).all()
    assert not np.isfinite(got[4]).any()


def test_same_bits_every_time():
    for T in (1, 16, 40, 300):
        codes, scales = make(700, 2048, 4, 128)
        x = acts(T, 2048)
        first = run(x, codes, scales, 4, 128)
        for _ in range(5):
            assert np.array_equal(run(x, codes, scales, 4, 128), first)


@pytest.mark.parametrize("bits", [4, 8])
def test_quantized_from_fp16(bits):
    """The codes and scales of the framework's own quantize call."""
    import torch
    import int4_grouped_expert_gb300 as st
    w = gen.expert_weight(0, 0, 1, "gate", 200, 512)
    lin = st.QuantLinear.from_fp16(torch.from_numpy(w), bits=bits)
    codes = lin.codes.cpu().numpy().view(np.uint8)
    x = acts(9, 512)
    got = run(x, codes, lin.scales.cpu().numpy(), bits, 128)
    y = ref.bf16_bits_to_f64(x) @ w.astype(np.float64).T
    # a code is off by at most half a scale: uniform, 1/sqrt(12) of a scale in the mean per weight
    s = lin.scales.cpu().numpy().astype(np.float64).max()
    assert np.abs(got - y).max() < 6 * s / np.sqrt(12) * np.sqrt(512) + 0.01



@pytest.mark.parametrize("T", [33, 64, 65, 200, 513])
@pytest.mark.parametrize("N", [8, 100, 256, 1030])
@pytest.mark.parametrize("bits", [4, 8])
def test_few_weights_for_many_tokens(T, N, bits):
    """Small matrices are streamed for longer batches than large ones."""
    check(T, N, 512, bits, 128, with_bias=True, with_res=True)


@pytest.mark.parametrize("bits,group", [(4, 64), (4, 128), (4, 256), (8, 64), (8, 128), (8, 256)])
@pytest.mark.parametrize("T", [33, 64, 65, 130, 257])
def test_every_format_and_batch_of_a_wide_layer(T, bits, group):
    check(T, 5003, 768, bits, group)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("K,group", [(64, 64), (192, 64), (128, 128), (384, 128), (1152, 128), (256, 256)])
@pytest.mark.parametrize("T", [40, 90])
def test_contraction_lengths_of_a_wide_layer(T, K, group, bits):
    check(T, 5003, K, bits, group)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,N", [(40, 1500), (61, 2100), (128, 1024), (250, 700)])
def test_long_contractions_are_shared(T, N, bits):
    """Few tiles and a long contraction: blocks share a tile, with bias, residual and odd rows."""
    check(T, N, 7168, bits, 128, with_bias=True, with_res=True, out_pad=5)
    check(T, N, 7168, bits, 64, with_bias=True, with_res=True, in_place=True)


@pytest.mark.parametrize("T,N,K", [(40, 5003, 256), (300, 5003, 256), (1100, 2049, 256), (3000, 1030, 128)])
def test_bias_residual_and_strides_of_a_wide_layer(T, N, K):
    """Several rounds of tiles, token tiles below the largest, rows at any alignment."""
    check(T, N, K, 4, 64, with_bias=True, with_res=True, x_pad=8, out_pad=3)
    check(T, N, K, 8, 128, with_bias=True, with_res=True, x_pad=40, out_pad=1, in_place=True)
