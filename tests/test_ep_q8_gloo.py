"""Expert parallelism with 8-bit rows on CPU, two gloo ranks: codes and scales
travel with their rows, so that a stand-in expert (the widened row times
expert id + 1) gives, bit for bit, what the same arithmetic gives without any
exchange; every rank receives its experts' rows only, and a rank without
tokens takes part."""
import os

import pytest
import torch
import torch.multiprocessing as mp

from bit_quantized_moe_softmax_b200 import dist as D
from bit_quantized_moe_softmax_b200 import ep
from tests.test_ep_gloo import _free_port, _rank_data


def _q8(x, dtype, columns):
    """Codes and scales of x as the norm's 8-bit output defines them."""
    n, H = x.shape
    qmax = 448.0 if dtype == torch.float8_e4m3fn else 127.0
    parts = x.split(columns or H, dim=1)
    scale = torch.stack([p.abs().amax(1) for p in parts], 1) / qmax if n else torch.zeros(0, len(parts))
    t = torch.cat([p / scale[:, i:i + 1] for i, p in enumerate(parts)], 1)
    return (t.round() if dtype == torch.int8 else t).to(dtype), scale


def _widen(q, scale, columns):
    return q.float() * scale.repeat_interleave(columns or q.shape[1], 1)[:, :q.shape[1]]


def _exchange(r, world, ns, dtype, columns):
    E, k, H = 8, 2, 80
    x, ids, w, base = _rank_data(r, ns[r], E, k, H)
    q, scale = _q8(x, dtype, columns)
    owner = ep.expert_owner(E, world)
    right = []

    def local_fn(codes, scales, eid):
        right.append(codes.dtype == dtype and bool((owner[eid] == r).all()))
        return _widen(codes, scales, columns) * (eid + 1).float()[:, None]

    out = ep.moe_forward_ep_q8(q, scale, ids, w, E, local_fn, base)
    ref, rows = base.clone(), _widen(q, scale, columns) if ns[r] else x
    for j in range(k):
        ref = torch.addcmul(ref, w[:, j:j + 1], rows * (ids[:, j] + 1).float()[:, None])
    return bool(torch.equal(out, ref)) and all(right)


def _worker(rank, world, port, q):
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port), RANK=str(rank), LOCAL_RANK=str(rank),
                      WORLD_SIZE=str(world))
    try:
        r, _, w = D.init("gloo", timeout_s=60)
        res = [_exchange(r, w, ns, t, c) for ns in ([5, 3], [4, 0]) for t in (torch.float8_e4m3fn, torch.int8)
               for c in (0, 32)]
        D.barrier()
        q.put((r, res))
        D.finish()
    except Exception as e:  # report instead of hanging the parent
        import traceback

        q.put(("error", traceback.format_exc() + repr(e)))


def test_expert_parallel_q8_gloo():
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    port = _free_port()
    procs = [ctx.Process(target=_worker, args=(r, 2, port, q)) for r in range(2)]
    for p in procs:
        p.start()
    got = [q.get(timeout=300) for _ in procs]
    for p in procs:
        p.join(timeout=60)
    assert all(g[0] != "error" and all(g[1]) for g in got), got


@pytest.mark.parametrize("columns", [0, 32])
def test_one_process(columns):
    assert _exchange(0, 1, [6], torch.int8, columns)
