"""Argument checks of the attention with first tokens, on the host before any CUDA call."""
from test_block_abi_cpu import A, batch, cache, st  # noqa: F401


def test_refusals(st):  # noqa: F811
    C, b = cache(st), batch(st)
    need = st.strata_attention_workspace_size(C, b, 32)
    ok = dict(workspace=A, ws_bytes=1 << 40)
    f = st.strata_attention_sinks_forward
    assert f(C, b, A, 32, 0.1, 2 * A, n_sinks=-1, **ok) == 1
    assert f(C, b, A, 32, 0.1, 2 * A, n_sinks=-1, window=9, **ok) == 1
    assert f(C, b, A, 32, 0.1, 2 * A, n_sinks=4, window=-1, **ok) == 1
    assert f(C, b, A, 32, float("nan"), 2 * A, window=9, n_sinks=4, **ok) == 1
    assert f(C, b, A, 32, 0.1, 2 * A, window=9, n_sinks=4, flags=1, **ok) == 1
    assert f(C, b, A, 12, 0.1, 2 * A, window=9, n_sinks=4, **ok) == 3
    assert f(C, b, A, 32, 0.1, A, window=9, n_sinks=4, **ok) == 1
    assert f(C, b, A, 32, 0.1, 2 * A, A, need - 1, window=9, n_sinks=4) == 4
    assert f(C, batch(st, max_kv=513), A, 32, 0.1, 2 * A, window=9, n_sinks=4, **ok) == 2
    assert f(C, batch(st, T=0), A, 32, 0.1, 2 * A, None, 0, window=9, n_sinks=4) == 0
