"""What a projection rounds: nothing up to LINEAR_EXACT_T tokens, beyond that each weight once to f16
(2^-11 of itself). The bound here follows that promise, tightly enough that bf16 weights fail it."""
import numpy as np
import pytest

import block_ref as ref
from test_gpu_linear import acts, make, run
from workloads import gen

EXACT_T = 64


def bound(x, codes, scales, bits, group, T):
    """The sum in 64 bits and the error allowed to a bf16 result. fp32 sums: 32 units in the last place of
    the sum of magnitudes (tens of additions to a partial sum, random in sign). f16 weights: each is
    off by up to 2^-11 of itself, so by 2^-11 / sqrt(3) in the mean at most, and the sum by that times
    ||x w||_2: 4 * 2^-11 is seven of those. f16 activations: 2^-25 of the power of two that brings a row's
    largest below 16, for entries below 2^-14 of that. The output's own rounding: half a unit."""
    w = ref.unpack(codes, bits) * np.repeat(scales.astype(np.float64), group, axis=1)
    y = x @ w.T
    b = 32 * ref.U32 * (np.abs(x) @ np.abs(w).T)
    if T > EXACT_T:
        b += 4 * 2.0 ** -11 * np.sqrt((x * x) @ (w * w).T)
        b += 2.0 ** -28 * np.abs(x).max(1, keepdims=True) * np.abs(w).sum(1)[None]
    return y, b + ref.half_ulp_bf16(np.abs(y) + b)


def worst(got, x, codes, scales, bits, group):
    y, b = bound(x, codes, scales, bits, group, len(x))
    return (np.abs(got - y) / b).max()


FORMATS = [(4, 64), (4, 128), (4, 256), (8, 64), (8, 128), (8, 256)]


def rounded(x, w, kind):
    """The projection with weights rounded to 8 (bf16) or 11 (f16) bits, and the output to bf16."""
    if kind == "f16":
        w = w.astype(np.float16).astype(np.float64)
    else:
        w = ref.bf16_bits_to_f64(gen.f32_to_bf16_bits(w.astype(np.float32)))
    return ref.bf16_bits_to_f64(gen.f32_to_bf16_bits((x @ w.T).astype(np.float32)))


@pytest.mark.parametrize("bits,group", FORMATS)
def test_the_bound_holds_f16_weights_and_refuses_bf16_ones(bits, group):
    codes, scales = make(145, 768, bits, group)
    x = ref.bf16_bits_to_f64(acts(200, 768))
    w = ref.unpack(codes, bits) * np.repeat(scales.astype(np.float64), group, axis=1)
    assert worst(rounded(x, w, "f16"), x, codes, scales, bits, group) < 1
    assert worst(rounded(x, w, "bf16"), x, codes, scales, bits, group) > 1.5


def test_the_threshold_is_the_library_s():
    import int4_grouped_expert_gb300 as st
    assert st.LINEAR_EXACT_T == EXACT_T


@pytest.mark.gpu
@pytest.mark.parametrize("bits,group", FORMATS)
@pytest.mark.parametrize("T,N,K", [(33, 5003, 768), (64, 5003, 768), (64, 145, 768), (65, 5003, 768), (130, 2100, 768),
                                   (200, 5003, 512), (300, 1500, 7168), (1100, 1030, 1024)])
def test_every_format(T, N, K, bits, group):
    codes, scales = make(N, K, bits, group)
    x = acts(T, K)
    w = worst(run(x, codes, scales, bits, group), ref.bf16_bits_to_f64(x), codes, scales, bits, group)
    print(f"worst error / bound {w:.3f}")
    assert w <= 1


@pytest.mark.gpu
@pytest.mark.parametrize("T", [40, 64, 96, 200])
@pytest.mark.parametrize("N", [64, 5003])
def test_large_and_small_activations(T, N):
    """Rows far outside the f16 range on either side keep their relative precision."""
    codes, scales = make(N, 512, 4, 128)
    x = ref.bf16_bits_to_f64(acts(T, 512)) * np.exp2(np.linspace(-40, 40, T).round())[:, None]
    bits = gen.f32_to_bf16_bits(x.astype(np.float32))
    assert worst(run(bits, codes, scales, 4, 128), ref.bf16_bits_to_f64(bits), codes, scales, 4, 128) <= 1


@pytest.mark.gpu
@pytest.mark.parametrize("T", [50, 90])
@pytest.mark.parametrize("N", [100, 5003])
def test_non_finite_rows_stay_alone(T, N):
    codes, scales = make(N, 512, 8, 128)
    scales[37, 2] = np.nan
    x = acts(T, 512)
    x[2, 11], x[4, 100] = 0x7FC0, 0x7F80                                  # a nan and an inf
    got = run(x, codes, scales, 8, 128)
    rows, cols = np.delete(np.arange(T), [2, 4]), np.delete(np.arange(N), 37)
    assert np.isnan(got[2]).all() and np.isnan(got[:, 37]).all() and not np.isfinite(got[4]).any()
    y, b = bound(ref.bf16_bits_to_f64(x[rows]), codes[cols], scales[cols], 8, 128, T)
    assert (np.abs(got[np.ix_(rows, cols)] - y) <= b).all()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T", [9, 16])
@pytest.mark.parametrize("N,K", [(4864, 1536), (4865, 1408), (4865, 1536), (5003, 3200), (7296, 2944), (7297, 3200)])
def test_blocks_of_a_wide_layer(T, N, K, bits):
    """Both sides of the sizes at which blocks change their shape."""
    codes, scales = make(N, K, bits, 128)
    x = acts(T, K)
    assert worst(run(x, codes, scales, bits, 128), ref.bf16_bits_to_f64(x), codes, scales, bits, 128) <= 1
