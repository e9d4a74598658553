"""Argument checks of the sampling call (on the CPU: before any launch)."""
from test_kv_host import DEV, w12  # noqa: F401


def test_refusals(w12):  # noqa: F811
    E, L = w12, w12.lib()

    def sample(lg=DEV, dt=0, R=2, T=3, V=100, temp=DEV, k=DEV, p=DEV, m=DEV, u=DEV, tok=DEV, prob=DEV, draft=DEV,
               acc=DEV, nxt=DEV, ws=DEV, wsb=512):
        return L.w12_sample(lg, dt, R, T, V, temp, k, p, m, u, tok, prob, draft, acc, nxt, ws, wsb, None)

    for kw, want in [(dict(dt=2), E.ERR_ARG), (dict(R=0), E.ERR_SHAPE), (dict(T=0), E.ERR_SHAPE),
                     (dict(V=0), E.ERR_SHAPE), (dict(V=E.SAMPLE_MAX_V + 1), E.ERR_SHAPE),
                     (dict(R=1 << 20, T=1 << 7), E.ERR_SHAPE), (dict(lg=None), E.ERR_ARG), (dict(u=None), E.ERR_ARG),
                     (dict(tok=None), E.ERR_ARG), (dict(acc=None), E.ERR_ARG), (dict(nxt=None), E.ERR_ARG),
                     (dict(draft=None), E.ERR_ARG), (dict(lg=DEV + 2), E.ERR_ALIGN),
                     (dict(lg=DEV + 1, dt=1), E.ERR_ALIGN), (dict(temp=DEV + 2), E.ERR_ALIGN),
                     (dict(k=DEV + 1), E.ERR_ALIGN), (dict(prob=DEV + 2), E.ERR_ALIGN),
                     (dict(ws=None), E.ERR_WORKSPACE), (dict(wsb=511), E.ERR_WORKSPACE), (dict(ws=DEV + 16), E.ERR_ALIGN)]:
        assert sample(**kw) == want, kw
    assert L.w12_sample_workspace_size(0, 1, 10) == 0
    assert L.w12_sample_workspace_size(1, 1, E.SAMPLE_MAX_V + 1) == 0
    assert L.w12_sample_workspace_size(1, 1, E.SAMPLE_MAX_V) == 512
