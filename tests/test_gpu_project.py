"""ds4moe_project against the formula in 64 bits.

Bound of an output, derived from the arithmetic: half a step of bf16 (2^-8 of
the value) for the one rounding at the end; the accumulation in binary32, where
each of the K / 16 steps of the matrix unit may drop up to two units in the last
place of a partial sum, at most 2^-22 K / 16 times the sum of the products'
magnitudes (the first product of the adapters alike, and 2^-22 for the sums over
its eight warps and eight CTAs); t = scale A x enters the second product with 16
bits (2^-16 of it).
"""
import pytest
import torch

import bit_quantized_moe_softmax_b200 as m
from bit_quantized_moe_softmax_b200 import synth
from tests.test_gpu_sample import reference as sample_reference

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_quantized_moe_softmax_b200 import build

    build.build()


def _data(n, fin, fout, na, rank, ids="mixed", seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 31 * n + fin + fout + rank)

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda")

    d = dict(x=randn(n, fin).to(BF16), W=(randn(fout, fin) * fin ** -0.5).to(BF16))
    if na:
        d["A"] = (randn(na, rank, fin) * fin ** -0.5).to(BF16)
        d["B"] = (randn(na, fout, rank) * rank ** -0.5).to(BF16)
        d["adapter_scale"] = torch.rand(na, generator=g, device="cuda") * 2 - 0.5
        i = torch.arange(n, device="cuda")
        d["ids"] = {"mixed": torch.randint(-1, na, (n,), generator=g, device="cuda"), "own": i % na,
                    "runs": (i * min(na, 5) // max(n, 1)) % na, "one": torch.full((n,), na - 1, device="cuda"),
                    "none": torch.full((n,), -1, device="cuda"),
                    "wild": torch.where(i % 3 == 0, na + i, torch.where(i % 3 == 1, -7 - i, i % na))}[ids].to(torch.int32)
    return d


def _reference(d):
    """(out, bound) in 64 bits."""
    x, W = d["x"].double(), d["W"].double()
    n, fin = x.shape
    y = x @ W.t()
    size = x.abs() @ W.abs().t() * (fin / 16 + 1)
    t_err = torch.zeros_like(y)
    if "A" in d:
        for a in range(d["A"].shape[0]):
            at = torch.nonzero(d["ids"] == a)[:, 0]
            if at.numel():
                A, B, s = d["A"][a].double(), d["B"][a].double(), d["adapter_scale"][a].double()
                t = s * (x[at] @ A.t())
                y[at] += t @ B.t()
                t_size = s.abs() * (x[at].abs() @ A.abs().t())
                size[at] += t_size @ B.abs().t() * (fin / 16 + 32) + t.abs() @ B.abs().t() * 16
                t_err[at] += t.abs() @ B.abs().t() * 2.0 ** -16
    return y, y.abs() * 2.0 ** -8 + size * 2.0 ** -22 + t_err


def _check(d, **kw):
    n, fout = d["x"].shape[0], d["W"].shape[0]
    out = torch.full((n + 1, fout), 77.0, dtype=BF16, device="cuda")
    m.ds4moe_project(out=out[:n], **d, **kw)
    torch.cuda.synchronize()
    y, bound = _reference(d)
    err = (out[:n].double() - y).abs()
    assert bool((err <= bound).all()), ((err / bound).max().item(), (err / bound).argmax().item())
    assert bool((out[n] == 77).all()), "rows behind the last one"
    assert m.ds4moe_get_project_error() == 0
    return out[:n]


@pytest.mark.parametrize("n", [1, 2, 7, 8, 15, 16, 17, 33, 64, 65, 100, 128, 129, 200, 256, 257, 300])
@pytest.mark.parametrize("ids", ["mixed", "runs", "wild"])
def test_row_counts(n, ids):
    _check(_data(n, 512, 640, 5, 16, ids))


@pytest.mark.parametrize("fin", [8, 24, 64, 72, 128, 1032, 4096])
@pytest.mark.parametrize("n", [1, 20, 130])
def test_input_widths(n, fin):
    _check(_data(n, fin, 257, 3, 24))


@pytest.mark.parametrize("fout", [1, 2, 63, 127, 128, 129, 511, 513, 1000, 5001])
@pytest.mark.parametrize("n", [3, 40, 150])
def test_output_widths(n, fout):
    _check(_data(n, 256, fout, 3, 8))


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 72, 128])
@pytest.mark.parametrize("n", [2, 48, 160])
def test_ranks(n, rank):
    _check(_data(n, 320, 300, 4, rank))


@pytest.mark.parametrize("ids", ["own", "one", "none"])
@pytest.mark.parametrize("n, na", [(1, 1), (5, 70), (64, 64), (64, 1), (256, 200), (300, 300), (600, 3)])
def test_adapters_of_rows(n, na, ids):
    _check(_data(n, 256, 384, na, 16, ids))


@pytest.mark.parametrize("n, fin, fout", [(1, 64, 32768), (4, 4096, 4096), (64, 1024, 20000), (1000, 512, 4096),
                                          (2000, 1024, 2000), (1030, 264, 10007)])
@pytest.mark.parametrize("na", [0, 6])
def test_tile_plans(n, fin, fout, na):
    """Split tiles, many tiles per CTA, CTA pairs and their ragged edges, with and without adapters."""
    _check(_data(n, fin, fout, na, 32, "runs"))


def test_no_adapters_is_the_projection_alone():
    d = _data(70, 512, 300, 3, 8, "none")
    a = _check(d)
    b = _check(dict(x=d["x"], W=d["W"]))
    assert torch.equal(a, b)


def test_repeats_bitwise_and_does_not_mix_rows():
    """The same call twice gives the same bits, and a row's output does not depend on the other rows of its tile: with
    NaN and infinities in every other row of x, the rest stay as they were."""
    for n in (6, 40, 200):
        d = _data(n, 256, 300, 4, 16)
        a, b = _check(d), _check(d)
        assert torch.equal(a, b)
        bad = dict(d, x=d["x"].clone())
        bad["x"][1::2, 5] = float("nan")
        bad["x"][3::4, 9] = float("inf")
        out = torch.empty_like(a)
        m.ds4moe_project(out=out, **bad)
        assert torch.equal(out[0::2], a[0::2]) and bool(out[1::2].isnan().all())


def test_stream_graph_and_work_buffer():
    d = _data(48, 512, 640, 7, 16)
    ref = _check(d)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(ref)
    m.ds4moe_project(out=out, stream=st, **d)
    st.synchronize()
    assert torch.equal(out, ref)
    need = m.ds4moe_project_work_bytes(48, 512, 640, 7, 16)
    work = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")   # NaN bits: what is not written is not read
    g = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(g):
        m.ds4moe_project(out=out, work=work[:need], **d)
        m.ds4moe_project(out=out, work=work[:need], **d)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and bool((work[need:] == 255).all())
    for n in (3, 100):   # the other forms of the work buffer
        e = _data(n, 512, 640, 7, 16)
        need = m.ds4moe_project_work_bytes(n, 512, 640, 7, 16)
        work = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
        _check(e, work=work[:need])
        assert bool((work[need:] == 255).all())
    with pytest.raises(m.Ds4MoeError):
        m.ds4moe_project(out=out, work=work[:64], **d)


def test_own_work_buffers_of_several_streams():
    """Calls without a work buffer on two side streams and the current one, in turn: each has its own."""
    ds = [_data(n, 512, 640, 7, 16, seed=n) for n in (3, 48, 100)]
    refs = [_check(d) for d in ds]
    streams = [torch.cuda.Stream(), torch.cuda.Stream(), None]
    outs = [[torch.empty_like(r) for _ in range(12)] for r in refs]
    torch.cuda.synchronize()
    for i in range(12):
        for d, o, s in zip(ds, outs, streams):
            m.ds4moe_project(out=o[i], stream=s, **d)
    torch.cuda.synchronize()
    assert all(torch.equal(o, r) for os_, r in zip(outs, refs) for o in os_)


def test_refuses_overlaps_and_layouts():
    d = _data(8, 64, 64, 0, 0)
    with pytest.raises(m.Ds4MoeError):
        m.ds4moe_project(out=d["x"], **d)
    with pytest.raises(m.Ds4MoeError):
        m.ds4moe_project(x=d["x"].t().contiguous().t(), W=d["W"], out=torch.empty(8, 64, dtype=BF16, device="cuda"))
    with pytest.raises(m.Ds4MoeError):
        m.ds4moe_project(x=d["x"], W=d["W"].cpu(), out=torch.empty(8, 64, dtype=BF16, device="cuda"))


def test_one_decode_step_around_the_layer(orc):
    """From the residual stream to the next token: the layer on the normed rows, its output joining the stream, the
    last norm, the head with the requests' adapters, and sampling; each step checked on what it was given."""
    from tests._util import oracle_layer, pack_with_oracle, rel_err

    H, V, n, na = 256, 1000, 6, 3
    L = synth.float_layer(synth.Shape(H=H, I=128, E=8, k=2), 5)
    L.update(pack_with_oracle(orc, L))
    lay = m.MoELayer(H, 128, 8, 2, 8)
    lay.load(L)
    g = torch.Generator(device="cuda").manual_seed(9)
    stream = torch.randn(n, H, generator=g, device="cuda")
    w1, w2 = (torch.rand(H, generator=g, device="cuda") + 0.5 for _ in range(2))
    x = torch.empty(n, H, device="cuda")
    m.ds4moe_add_rmsnorm(stream, w1, 1e-6, out=x)
    y = lay.forward(x)
    ref, _, _ = orc.moe_forward(oracle_layer(L), x.cpu().numpy())
    assert rel_err(y.cpu(), ref) < 1e-4
    total = stream + y
    h = torch.empty(n, H, dtype=BF16, device="cuda")
    m.ds4moe_add_rmsnorm(y, w2, 1e-6, residual=stream, sum=stream, out=h)
    assert torch.equal(stream, total)
    d = _data(n, H, V, na, 16, "mixed", seed=4)
    d["x"], d["W"] = h, (d["W"].float() * 8).to(BF16)
    logits = _check(d)
    u = torch.rand(n, generator=g, device="cuda")
    p = dict(temperature=torch.full((n,), 0.8, device="cuda"), top_k=torch.full((n,), 50, dtype=torch.int32, device="cuda"),
             top_p=torch.full((n,), 0.9, device="cuda"), min_p=torch.full((n,), 0.02, device="cuda"))
    token, prob = torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(n, device="cuda")
    m.ds4moe_sample(logits, u, token, prob=prob, **p)
    for i in range(n):
        t, pr, _ = sample_reference(logits[i], float(u[i]), 0.8, 50, float(p["top_p"][i]), float(p["min_p"][i]))
        assert int(token[i]) == t and abs(float(prob[i]) - pr) < 1e-6
