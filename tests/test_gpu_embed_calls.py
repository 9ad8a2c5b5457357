"""What calls of the input-layer operators refuse, report and share: overlaps
with the places, empty places' positions, host threads, tensors that require a
gradient, sequence lengths."""
import threading

import numpy as np
import pytest

from tests import embed_reference as ref
from tests.test_gpu_embed import _check, _np, _rand, ops  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_results_over_the_places_are_refused(ops):
    """A result that shares bytes with the tokens or positions would change what the call still reads."""
    V, D, P = 100, 16, 8
    layer = ops.TokenEmbedding(V, D, 16, positions=P)
    table, wpe = _rand((V, D), "f32", 1).cuda(), _rand((P, D), "f32", 2).cuda()
    dout = torch.ones(2, 8, D, device="cuda")
    free = torch.zeros(2, 8, dtype=torch.int64, device="cuda")
    for at in (0, 40, 127):  # the first, an inner and the last 8 bytes of the 16 x 16 fp32 result
        buffer = torch.zeros(1024, dtype=torch.int64, device="cuda")
        over = buffer[at:at + 16].view(2, 8)
        out = buffer.view(torch.float32)[:256].view(2, 8, D)
        with pytest.raises(ops.LionCubError, match="out overlaps"):
            layer.forward(over, table, out=out)
        with pytest.raises(ops.LionCubError, match="out overlaps"):
            layer.forward(free, table, wpe, positions=over, out=out)
        grad = buffer.view(torch.float32)[:V * D].view(V, D)
        with pytest.raises(ops.LionCubError, match="grad overlaps"):
            layer.backward(over, dout, grad)
        spare = torch.empty(V, D, device="cuda")
        pos_grad = buffer.view(torch.float32)[:P * D].view(P, D)
        where = buffer[at % 64:at % 64 + 16].view(2, 8)
        with pytest.raises(ops.LionCubError, match="pos_grad overlaps"):
            layer.backward(where, dout, spare, pos_grad=pos_grad)
        with pytest.raises(ops.LionCubError, match="pos_grad overlaps"):
            layer.backward(free, dout, spare, pos_grad=pos_grad, positions=where)
        assert (buffer == 0).all()
    layer.close()


def test_places_beside_the_results_rows(ops):
    """Tokens that lie right before or behind a result, or in the gap between two of its rows, share nothing with it."""
    V, D = 50, 16
    layer = ops.TokenEmbedding(V, D, 8)
    table = _rand((V, D), "f32", 1).cuda()
    want = torch.randint(0, V, (8,), dtype=torch.int32, device="cuda")
    for at in (0, 8 + 16, 8 + 24 + 16, 8 + 7 * 24 + 16):
        buffer = torch.zeros(8 + 8 * 24, dtype=torch.int32, device="cuda")
        tok = buffer[at:at + 8]
        tok.copy_(want)
        out = buffer[8:].view(torch.float32).view(8, 24)[:, :D]
        layer.forward(tok, table, out=out)
        assert torch.equal(tok, want) and torch.equal(out, table[want.long()])
    layer.close()


@pytest.mark.parametrize("index", [torch.int64, torch.int32])
@pytest.mark.parametrize("n", [6, 3000])  # one place a warp, and several
def test_positions_of_empty_places_may_be_anything(ops, index, n):
    """Both arrays padded alike, with -1 or with numbers beyond the table."""
    V, P, D = 50, 10, 256
    rng = np.random.default_rng(n)
    tok, pos = rng.integers(0, V, n), rng.integers(0, P, n)
    tok[1::3] = -1
    pos[1::3] = np.where(np.arange(len(pos[1::3])) % 2, -1, P + 5)
    t, q = (torch.from_numpy(v).to(index).cuda() for v in (tok, pos))
    table, wpe, dout = _rand((V, D), "f32", 1), _rand((P, D), "f32", 2), _rand((n, D), "f32", 3)
    layer = ops.TokenEmbedding(V, D, n, positions=P)
    out = layer.forward(t, table.cuda(), wpe.cuda(), positions=q, out_dtype=torch.float32)
    assert layer.status() == 0
    want = torch.where(t[:, None] < 0, torch.zeros(1, device="cuda"),
                       table.cuda()[t.long().clamp(min=0)] + wpe.cuda()[q.long().clamp(0, P - 1)])
    assert torch.equal(out, want)
    grad, pos_grad = torch.empty(V, D, device="cuda"), torch.empty(P, D, device="cuda")
    layer.backward(t, dout.cuda(), grad, pos_grad=pos_grad, positions=q)
    assert layer.status() == 0
    token, position = ref.gradients(tok, V, P, _np(dout), 1.0, None, positions=pos)
    for got, (exact, mag, count) in ((grad, token), (pos_grad, position)):
        _check(got, exact, mag, count + 3, "f32")
    layer.close()


def _side_by_side(*work):
    """Runs the functions in threads of their own; what they raised."""
    raised = []

    def go(f):
        try:
            f()
        except Exception as e:  # noqa: BLE001
            raised.append(e)

    threads = [threading.Thread(target=go, args=(f,)) for f in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return raised


def test_layers_of_different_sizes_in_two_threads(ops):
    """Gradients of two layers whose sorts take different amounts of shared memory, from a host thread each."""
    D, n, calls = 8, 64, 4000

    def layer_of(V, seed):
        layer, stream = ops.TokenEmbedding(V, D, n), torch.cuda.Stream()
        tok = torch.randint(0, V, (n,), generator=torch.Generator().manual_seed(seed)).cuda()
        dout, grad = torch.ones(n, D, device="cuda"), torch.zeros(V, D, device="cuda")
        want = torch.zeros_like(grad).index_add_(0, tok, dout)
        torch.cuda.synchronize()

        def work():
            for _ in range(calls):
                layer.backward(tok, dout, grad, stream=stream)

        return work, layer, grad, want

    parts = [layer_of(1 << 20, 1), layer_of(600000, 2)]
    raised = _side_by_side(*(p[0] for p in parts))
    torch.cuda.synchronize()
    assert not raised, raised[0]
    for _, layer, grad, want in parts:
        assert torch.equal(grad, want) and layer.status() == 0
        layer.close()


def test_lookups_of_one_layer_in_several_threads(ops, monkeypatch):
    """Lookups share nothing: every launch is counted once (one of them is made to fail), results are each call's own."""
    V, D, threads, calls = 300, 64, 4, 2000
    monkeypatch.setenv("LIONCUB_FAIL_LAUNCH", str(threads * calls))
    layer = ops.TokenEmbedding(V, D, 64)
    monkeypatch.delenv("LIONCUB_FAIL_LAUNCH")
    table = _rand((V, D), "f32", 1).cuda()
    tokens = [torch.randint(0, V, (64,), device="cuda") for _ in range(threads)]
    outs = [torch.empty(64, D, device="cuda") for _ in range(threads)]
    torch.cuda.synchronize()

    def work(k):
        stream = torch.cuda.Stream()
        for _ in range(calls):
            layer.forward(tokens[k], table, out=outs[k], stream=stream)

    raised = _side_by_side(*(lambda k=k: work(k) for k in range(threads)))
    torch.cuda.synchronize()
    assert len(raised) == 1 and "launch" in str(raised[0]), raised
    for t, out in zip(tokens, outs):
        assert torch.equal(out, table[t])
    layer.close()


def test_messages_are_each_threads_own(ops):
    """What failed last in this thread, whatever failed on the handle elsewhere since; else what failed last."""
    from communication_compressed_sign_gb300 import embed
    L = embed.load()
    layer = ops.TokenEmbedding(10, 8, 4)
    other = ops.TokenEmbedding(10, 8, 4)
    batch = embed.TokenBatch(None, None, 5, 1, 0, 0, 0)  # more places than the layer's
    unknown = embed.TokenBatch(None, None, 0, 1, 0, 7, 0)

    def fail(b):
        import ctypes
        assert L.lioncub_embed_forward(layer.h, ctypes.byref(b), None, None, None, None, None) != 0

    message = lambda: L.lioncub_embed_last_error(layer.h).decode()  # noqa: E731
    assert message() == ""
    assert not _side_by_side(lambda: fail(batch))
    assert "places" in message()  # a thread without a failure of its own reads the handle's
    fail(batch)
    seen = []
    assert not _side_by_side(lambda: (fail(unknown), seen.append(message())))
    assert "index type 7" in seen[0] and "places" in message()
    assert L.lioncub_embed_last_error(other.h) == b""
    layer.close()
    other.close()


def test_tensors_that_require_a_gradient(ops):
    """Results are not part of torch's graph, so while it records, such tensors are refused rather than losing their
    gradient; without recording they are taken."""
    V, D, P = 20, 16, 4
    layer = ops.TokenEmbedding(V, D, 4, positions=P)
    tok = torch.arange(4, device="cuda").view(1, 4)
    free, leaf = torch.ones(V, D, device="cuda"), torch.ones(V, D, device="cuda", requires_grad=True)
    wpe = torch.ones(P, D, device="cuda", requires_grad=True)
    x = torch.ones(1, 4, D, device="cuda", requires_grad=True)
    drop = ops.Drop(0.5, 1)
    calls = [lambda: layer.forward(tok, leaf), lambda: layer.forward(tok, free, wpe), lambda: ops.dropout(x, drop),
             lambda: ops.dropout(x.detach(), drop, residual=x), lambda: ops.dropout_backward(x, drop),
             lambda: layer.backward(tok, x, free.clone()), lambda: layer.backward(tok, x.detach(), free.clone(), base=leaf)]
    for call in calls:
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
    with torch.no_grad():
        for call in calls:
            call()
    assert torch.equal(layer.forward(tok, leaf.detach(), out_dtype=torch.float32)[0], free[:4])
    layer.close()


def test_sequence_lengths_below_one(ops):
    V, D, P = 20, 16, 4
    layer = ops.TokenEmbedding(V, D, 4, positions=P)
    tok = torch.arange(4, device="cuda")
    table, wpe = torch.ones(V, D, device="cuda"), torch.ones(P, D, device="cuda")
    for seq_len in (0, -3):
        with pytest.raises(ops.LionCubError, match="positions"):
            layer.forward(tok, table, wpe, seq_len=seq_len)
        with pytest.raises(ops.LionCubError, match="positions"):
            layer.backward(tok, table[:4], table.clone(), pos_grad=wpe.clone(), seq_len=seq_len)
    assert layer.forward(torch.empty(3, 0, dtype=torch.int64, device="cuda"), table, wpe).shape == (3, 0, D)
    layer.close()
