"""The draft-and-verify example on the GPU: the projections, the cache, the attention and the verification
together, against a plain FP32 model on the dequantised weights."""
import pytest

import weight_only_bit_gb300 as w4

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def plain_logits(s, tokens):
    """The model in FP32 torch operations: dequantised weights, an exact cache, a full causal softmax."""
    from weight_only_bit_gb300.serve import HEAD_DIM as D, KV_HEADS, Q_HEADS

    def weight(layer, proj):
        packed, scales, n, k = s.weights[(layer, proj)]
        out = torch.empty((n, k), device=s.dev)
        w4.check(w4.w4_dequantize_nf4(packed, scales, s.code, out, n, k, s.bs))
        return out

    def norm(h):
        return (h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6)).half().float()

    def turn(x, heads):
        x = x.view(n, heads, D)
        c, t = s.cos[:n, None], s.sin[:n, None]
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * c - b * t, b * c + a * t], -1)

    n = len(tokens)
    h = s.embed[torch.tensor(tokens, device=s.dev)].float()
    mask = torch.ones((n, n), device=s.dev).tril().bool()
    for layer in range(s.layers):
        x = norm(h)
        q, k = turn(x @ weight(layer, "q").T, Q_HEADS), turn(x @ weight(layer, "k").T, KV_HEADS)
        v = (x @ weight(layer, "v").T).view(n, KV_HEADS, D)
        g = Q_HEADS // KV_HEADS
        k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
        p = torch.einsum("ihd,jhd->hij", q, k) * D ** -0.5
        p = p.masked_fill(~mask, float("-inf")).softmax(-1)
        o = torch.einsum("hij,jhd->ihd", p, v).reshape(n, -1)
        h = h + o @ weight(layer, "o").T
        x = norm(h)
        gate, up = x @ weight(layer, "gate").T, x @ weight(layer, "up").T
        h = h + (gate * torch.sigmoid(gate) * up) @ weight(layer, "down").T
    return norm(h) @ weight(*s.head).T


@pytest.fixture(scope="module")
def server(libw4):
    from weight_only_bit_gb300.serve import Server
    return Server(layers=2, capacity=256, page_tokens=32, drafts=4)


def reset(s):
    s.context, s.cached, s.steps, s.accepted = [], 0, 0, 0


def test_forward_matches_a_plain_model(server):
    """E4M3 keys and values are within 2^-4 of themselves, on average within 2^-5.2 (a value's place between
    two neighbours is uniform), and enter beside exact terms: the logits are within 5 % in the 2-norm, in
    one piece and in chunks."""
    s = server
    tokens = torch.randint(0, s.vocab, (70,), generator=torch.Generator().manual_seed(3)).tolist()
    want = plain_logits(s, tokens)
    for pieces in ([70], [1] * 5 + [33, 2, 30], [64, 5, 1]):
        reset(s)
        got, at = [], 0
        for n in pieces:
            got.append(s.forward(tokens[at:at + n]))
            at += n
        got = torch.cat(got).float()
        assert torch.isfinite(got).all()
        assert float((got - want).norm() / want.norm()) < 0.05
        # the last row by itself: an error in a later chunk cannot hide in the others
        assert float((got[-1] - want[-1]).norm() / want[-1].norm()) < 0.1
    w4.check(w4.w4_device_check())


def check_choices(s, prompt, out):
    """Every token of `out` is the argmax of the logits that the model gives when the same tokens are fed one
    after the other, up to the FP16 rounding of projections whose sums run in another order (the GEMVs
    agree with the exact product within 2e-2 of the root mean square; two of them and a norm)."""
    reset(s)
    s.forward(prompt[:-1])
    for prev, tok in zip([prompt[-1]] + out[:-1], out):
        row = s.forward([prev])[0].float()
        assert float(row.max() - row[tok]) <= 6e-2 * float(row.square().mean().sqrt())


def test_greedy_steps_emit_the_models_own_choices(server, monkeypatch):
    """With drafts from the context (nearly all refused: the model is random), and with the model's own next
    tokens as drafts (accepted), and what refused drafts leave behind in the cache does no harm."""
    s = server
    base = torch.randint(0, s.vocab, (12,), generator=torch.Generator().manual_seed(4)).tolist()
    prompt = base * 4                                 # repeats: lookups find drafts from the first step on
    reset(s)
    out = s.generate(prompt, 40)
    assert s.cached == len(s.context) - 1 and s.context[:len(prompt)] == prompt and s.context[len(prompt):][:40] == out
    assert len(s.context) - len(prompt) == s.steps + s.accepted
    check_choices(s, prompt, out)

    def ahead():                                      # three right drafts and a wrong one
        at = len(s.context) - len(prompt)
        return out[at:at + 3] + [(out[at] + 1) % s.vocab] if s.context[len(prompt):] == out[:at] else []

    reset(s)
    monkeypatch.setattr(s, "lookup", ahead)
    again = s.generate(prompt, 36)
    assert s.accepted >= 18 and s.steps <= 18         # about four tokens a step where the choices are clear
    check_choices(s, prompt, again)


def test_sampling_steps_stay_in_the_vocabulary(server):
    s = server
    reset(s)
    s.temperature = 0.7
    try:
        out = s.generate(torch.randint(0, s.vocab, (20,), generator=torch.Generator().manual_seed(5)).tolist(), 20)
        assert len(out) == 20 and all(0 <= t < s.vocab for t in out)
        with pytest.raises(w4.W4Error):
            s.forward([1] * 400)                      # beyond the cache
    finally:
        s.temperature = 0.0
