"""Host-side checks of the paged operators (no GPU): what the C entry points and the binding refuse."""
import pytest
import torch

import quantized_kv_cache_sm_gb300 as fa

P = 1 << 20   # a 16-byte aligned fake device address; never dereferenced by these calls
T = P + 256

ROWS = dict(k=P, v=P, kp=P, vp=P, table=T, starts=T, lens=T, B=2, rows=10, Hkv=2, D=128, NP=16,
            page=16, pps=8, krs=256, khs=128, vrs=256, vhs=128, dtype=0, kf=0, vf=0)
PREFILL = dict(q=P, kp=P, vp=P, o=P, table=T, starts=T, lens=T, B=2, rows=10, Hq=8, Hkv=2, D=128,
               NP=16, page=16, pps=8, qrs=1024, qhs=128, ors=1024, ohs=128, causal=1, scale=0.1,
               dtype=0, kf=0, vf=0, ws=P, wsb=1 << 40)
INV, UNS = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED

SHARED = [
    (dict(table=None), INV), (dict(starts=T + 2), INV), (dict(lens=None), INV),
    (dict(B=0), INV), (dict(rows=-1), INV), (dict(Hkv=0), INV), (dict(NP=0), INV),
    (dict(page=0), INV), (dict(pps=0), INV), (dict(B=1 << 17), INV), (dict(dtype=2), INV),
    (dict(kf=5), INV), (dict(vf=-1), INV), (dict(kp=P + 8), INV), (dict(vp=P + 8), INV),
    (dict(D=48), UNS), (dict(page=1 << 16, pps=1 << 15), UNS),
    (dict(NP=1 << 30, Hkv=2), UNS), (dict(NP=1 << 29, page=1 << 12), UNS),
]


@pytest.mark.parametrize("change,status", SHARED + [
    (dict(k=None), INV), (dict(v=None), INV), (dict(vp=None), INV), (dict(k=P + 4), INV),
    (dict(krs=100), INV), (dict(khs=-128), INV), (dict(vrs=1 << 41), INV), (dict(D=0), INV),
])
def test_rows_refusals(built, change, status):
    lib = built.load()
    a = {**ROWS, **change}
    k, v, kp, vp = a.pop("k"), a.pop("v"), a.pop("kp"), a.pop("vp")
    rest = list(a.values())
    assert lib.fa_append_paged(k, v, kp, vp, *rest, None) == status
    assert lib.fa_read_paged(kp, vp, k, v, *rest, None) == status


@pytest.mark.parametrize("krs,khs", [(0, 128), (256, 0), (128, 128), (128, 640), (64, 10000)])
def test_read_refuses_overlapping_outputs(built, krs, khs):
    lib = built.load()
    a = {**ROWS, "krs": krs, "khs": khs}
    k, v, kp, vp = a.pop("k"), a.pop("v"), a.pop("kp"), a.pop("vp")
    assert lib.fa_read_paged(kp, vp, k, v, *a.values(), None) == INV


@pytest.mark.parametrize("change,status", SHARED + [
    (dict(q=None), INV), (dict(o=P + 2), INV), (dict(vp=None), INV), (dict(Hq=7), INV),
    (dict(Hq=0), INV), (dict(scale=0.0), INV), (dict(scale=float("inf")), INV),
    (dict(qrs=100), INV), (dict(ors=0), INV), (dict(ohs=1024), INV), (dict(ws=None), INV),
    (dict(ws=P + 4), INV), (dict(D=96), UNS), (dict(page=24), UNS),
    (dict(Hq=258, qrs=258 * 128, ors=258 * 128), UNS),
])
def test_prefill_refusals(built, change, status):
    lib = built.load()
    assert lib.fa_prefill_paged(*{**PREFILL, **change}.values(), None) == status


def test_short_workspace_refused(built):
    lib = built.load()
    need = lib.fa_prefill_paged_workspace_bytes(8, 2, 128)
    if need == 0:
        pytest.skip("no device to size the scratch")
    assert lib.fa_prefill_paged(*{**PREFILL, "wsb": need - 1}.values(), None) == INV


def test_nothing_to_do(built):
    lib = built.load()
    assert lib.fa_append_paged(None, None, P, P, *list({**ROWS, "rows": 0}.values())[4:],
                               None) == fa.FA_OK
    assert lib.fa_prefill_paged(*{**PREFILL, "rows": 0, "q": None, "o": None}.values(),
                                None) == fa.FA_OK
    assert lib.fa_prefill_paged_workspace_bytes(8, 3, 128) == 0
    assert lib.fa_prefill_paged_workspace_bytes(8, 2, 96) == 0


def test_binding_refusals():
    """Raised before the library is called: shapes, dtypes, layouts, host tensors."""
    h = torch.float16
    q, pool = torch.zeros(5, 8, 128, dtype=h), torch.zeros(4, 2, 16, 128, dtype=h)
    kn = torch.zeros(5, 2, 128, dtype=h)
    i32 = dict(dtype=torch.int32)
    batch = (torch.zeros(2, 3, **i32), torch.zeros(3, **i32), torch.zeros(2, **i32))
    bad = [
        (ValueError, lambda: fa.fa_prefill_paged(q[0], pool, pool, *batch)),
        (ValueError, lambda: fa.fa_prefill_paged(q, pool, None, *batch)),
        (ValueError, lambda: fa.fa_prefill_paged(q[..., :64], pool, pool, *batch)),
        (ValueError, lambda: fa.fa_prefill_paged(q, pool, pool[:3], *batch)),
        (TypeError, lambda: fa.fa_prefill_paged(q.bfloat16(), pool, pool, *batch)),
        (TypeError, lambda: fa.fa_prefill_paged(q, pool, pool, *batch, q.bfloat16())),
        (ValueError, lambda: fa.fa_prefill_paged(q, pool, pool, *batch, q[:4])),
        (ValueError, lambda: fa.fa_prefill_paged(q, pool, pool, batch[0], batch[1][:2], batch[2])),
        (ValueError, lambda: fa.fa_prefill_paged(q, pool, pool, batch[0].long(), *batch[1:])),
        (ValueError, lambda: fa.fa_prefill_paged(q, pool, pool, *batch)),  # host tensors
        (ValueError, lambda: fa.fa_append_paged(kn, None, pool, pool, *batch)),
        (ValueError, lambda: fa.fa_append_paged(kn, kn[:4], pool, pool, *batch)),
        (TypeError, lambda: fa.fa_append_paged(kn, kn.bfloat16(), pool, pool, *batch)),
        (ValueError, lambda: fa.fa_append_paged(kn.mT.contiguous().mT, kn, pool, pool, *batch)),
        (ValueError, lambda: fa.fa_append_paged(kn, kn, pool, pool, *batch)),  # host tensors
        (ValueError, lambda: fa.fa_read_paged(pool, pool, *batch, kn)),
        (TypeError, lambda: fa.fa_read_paged(pool, None, *batch, kn.float())),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()


def test_workspace_that_does_not_hold_its_elements_is_refused():
    """An expanded tensor has as many elements as asked for and memory for one."""
    h, i32 = torch.float16, dict(dtype=torch.int32)
    q, pool = torch.zeros(5, 8, 128, dtype=h), torch.zeros(4, 2, 16, 128, dtype=h)
    batch = (torch.zeros(2, 3, **i32), torch.zeros(3, **i32), torch.zeros(2, **i32))
    ws = torch.zeros(1, dtype=torch.uint8).expand(1 << 40)
    with pytest.raises(ValueError, match="contiguous"):
        fa.fa_prefill_paged(q, pool, pool, *batch, workspace=ws)
