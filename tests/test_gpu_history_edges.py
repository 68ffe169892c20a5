"""Item ids and decay attention where they can go wrong, through the public
calls: the number of roundings of a bf16 call, timestamps that decrease, and
what a caller may do with streams, states and workspaces.

u16 = 2^-8 and u32 = 2^-24 are half a step of bf16 and fp32, M the same sum with
every term by its absolute value.
"""
import threading

import numpy as np
import pytest
import torch

import shared_prefix_behavior_b200 as R
import workloads as W
from oracle import rest_oracle as O
from tests.test_gpu_history import DT, U16, U32, _case, _dev

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- precision


def _rounded_once(got, want, mag, L, hd, what):
    """A bf16 result is the fp32 sum rounded once. The sum: (L + 2 head_dim + 64)
    u32 M as for an fp32 call, and a term passes at most two of the products whose
    operand is two bf16 numbers (its decayed key, the state), each off by 2^-16 of
    it; 2 % cover their second order. So, with s that bound, |got - want| <= s +
    u16 (|want| + s). The rounding of a value that is off by a small s is off
    from the exact value by little more than the exact value's own rounding:
    with s independent of it their squares add, and s is at most 2^-16 of a
    result that adds up like its terms, 2^-7 of what u16 leaves; the 2-norm may
    therefore exceed that rounding's by 2 %."""
    got = got.float().cpu().numpy().astype(np.float64)
    s = ((L + 2 * hd + 64) * U32 + 1.02 * 2 * 2.0 ** -16) * mag
    err = np.abs(got - want)
    assert np.all(err <= s + U16 * (np.abs(want) + s)), what
    rounding = np.linalg.norm(W.round_bf16(want).astype(np.float64) - want)
    assert np.linalg.norm(err) <= 1.02 * rounding, (what, float(np.linalg.norm(err) / rounding))


@pytest.mark.parametrize("hd,lengths", [(16, (700, 64, 129)), (32, (300,) * 90), (32, (1500, 1, 200)), (64, (1500, 65)),
                                        (64, (200, 330) * 20)])
def test_decay_bf16_results_are_rounded_once(cuda, hd, lengths):
    """Histories in one segment and in several; forward, with a state, and the gradients."""
    (q, k, v, d_o), ts, cu, taus, decay = _case("bf16", hd, lengths, 7 + hd)
    heads = R.DecayHeads(taus, decay, hd)
    t, tts, L = [_dev(x, "bf16") for x in (q, k, v, d_o)], torch.from_numpy(ts).to(cuda), max(lengths)
    want, _ = O.decay_attention(q, k, v, ts, cu, taus, decay)
    mag, _ = O.decay_attention(q, k, v, ts, cu, taus, decay, magnitude=True)
    _rounded_once(R.decay_attn_forward(*t[:3], cu, heads, ts=tts), want, mag, L, hd, "o")
    state = R.DecayState(heads, len(lengths), device=cuda)
    _rounded_once(R.decay_attn_forward(*t[:3], cu, heads, ts=tts, state=state), want, mag, L, hd, "o with a state")
    ref = O.decay_attention_backward(q, k, v, ts, cu, taus, decay, d_o)
    big = O.decay_attention_backward(q, k, v, ts, cu, taus, decay, d_o, magnitude=True)
    for name, g, r, m in zip(("dq", "dk", "dv"), R.decay_attn_backward(*t, cu, heads, ts=tts), ref, big):
        _rounded_once(g, r, m, L, hd, name)


# ---------------------------------------------------------------- timestamps that decrease


def test_decay_step_counts_a_decrease_as_no_time(cuda):
    """Factor 1 over the decrease, also to a time before the history's first; what follows counts from there."""
    heads = R.DecayHeads((1, 60), (-0.01, -0.5), 16)
    state = R.DecayState(heads, 1, device=cuda)
    hot = torch.zeros(5, 2, 16, device=cuda)
    hot[torch.arange(5), :, torch.arange(5)] = 1.0
    one = torch.zeros(1, 2, 16, device=cuda)
    one[:, :, 0] = 1.0
    err, seen = torch.zeros(1, dtype=torch.int32, device=cuda), []
    ts = [1000, 2000, 1500, 900, 1025]
    for i, t in enumerate(ts):
        R.decay_attn_step(one.view(1, 32), one.view(1, 32), hot[i:i + 1].view(1, 32), state, check=False, err=err,
                          ts=torch.tensor([t], device=cuda))
        seen.append(int(err))
    assert seen == [0, 0, 2, 2, 0] and state.t_last.item() == 1025 and state.t_first.item() == 1000
    for h, (tau, g) in enumerate(((1, -0.01), (60, -0.5))):
        n = [(t - 1000) // tau for t in ts]
        gaps = [max(0, b - a) for a, b in zip(n, n[1:])]
        for j in range(5):
            want = np.exp(g * sum(gaps[j:]))
            assert abs(float(state.s[0, h, 0, j]) - want) <= 8 * U32 * want


def _times(pattern, T):
    """Seconds since the history's first token, which decrease somewhere."""
    i = np.arange(T)
    if pattern == "steps":        # whole sixteens, up and down by hundreds of buckets
        return np.array([0, 1000, 500, 2000, 700])[i // 16 % 5]
    if pattern == "inside":       # within every sixteen, its last row the latest
        return np.array([0, 0, 0, 1000] + [10] * 11 + [1000])[i % 16]
    if pattern == "far inside":   # its first row further from its last than a middle one's decay can say
        return np.array([75] * 4 + [0] * 4 + [130] * 8)[i % 16]
    if pattern == "blocks":       # at the 64th row
        return 30 * (i % 64) + i // 64
    if pattern == "below":        # before the first token, by buckets and parts of them
        return np.where(i < 20, 7 * i, 5 * i - 1234)
    if pattern == "years":
        return np.where(i % 50 == 25, 10 ** 9, 100 * (i // 50)) + i
    return np.random.default_rng(5).integers(0, 3000, T)


def _weights(cuda, dtype, hd, heads, cu, ts, lo, hi, others, rng_seed=1):
    """The factor by which row j counts in row i of the history lo .. hi - 1, read
    off every output of the calls, {name: [n_heads, n, n]} and, from the state,
    [n_heads, n] for the last row: one-hot rows in one operand, constant ones in
    the others, whose products are exact. The other histories have the rows
    ``others``; what they give is returned too."""
    H, T, n = heads.n_heads, int(cu[-1]), hi - lo
    tts = torch.from_numpy(ts).to(cuda)
    one = torch.zeros(n, H, hd, device=cuda)
    one[:, :, 0] = 1.0
    root = float(hd) ** 0.5                       # 4 or 8: exact
    W4 = {name: torch.zeros(H, n, n, device=cuda) for name in ("o", "o with a state", "dq", "dk", "dv")}
    left, rest = torch.zeros(H, n, device=cuda), []

    def rows(x):
        full = others.clone()
        full[lo:hi] = x.reshape(n, H * hd).to(full.dtype)
        return full

    for b in range(0, n, hd):
        m = min(hd, n - b)
        hot = torch.zeros(n, H, hd, device=cuda)
        hot[torch.arange(b, b + m), :, torch.arange(m)] = 1.0
        state = R.DecayState(heads, len(cu) - 1, device=cuda)
        q, k, v = rows(one * root), rows(one), rows(hot)
        kw = dict(ts=tts, check=False)
        o = [R.decay_attn_forward(q, k, v, cu, heads, **kw), R.decay_attn_forward(q, k, v, cu, heads, state=state, **kw)]
        g = [R.decay_attn_backward(rows(one), rows(hot), rows(one), rows(one * root), cu, heads, **kw),
             R.decay_attn_backward(rows(hot), rows(one), rows(one), rows(one * root), cu, heads, **kw),
             R.decay_attn_backward(rows(one * root), rows(one), rows(one), rows(hot), cu, heads, **kw)]
        for name, x in (("o", o[0]), ("o with a state", o[1]), ("dq", g[0][0])):
            W4[name][:, :, b:b + m] = x[lo:hi].float().view(n, H, hd).permute(1, 0, 2)[:, :, :m]
        for name, x in (("dk", g[1][1]), ("dv", g[2][2])):
            W4[name][:, b:b + m, :] = x[lo:hi].float().view(n, H, hd).permute(1, 2, 0)[:, :m, :]
        u = [int(x) for x in cu].index(lo)
        left[:, b:b + m] = state.s[u, :, 0, :m]
        rest += [x[r] for x in (*o, *g[0]) for r in (slice(0, lo), slice(hi, T))]
        rest += [state.s[w] for w in range(len(cu) - 1) if w != u]
    return {name: w.cpu().numpy().astype(np.float64) for name, w in W4.items()}, left.cpu().numpy().astype(np.float64), rest


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decay_weights_over_a_far_decrease(cuda, dtype):
    """Hundreds of half-lives back: every factor stays between 0 and 1, also in the state."""
    cu = np.array([0, 200], dtype=np.int32)
    heads = R.DecayHeads((1, 60), (-0.7, -0.9), 16)
    ts = 10 ** 9 + _times("steps", 200).astype(np.int64)
    got, left, _ = _weights(cuda, dtype, 16, heads, cu, ts, 0, 200, torch.zeros(200, 32, device=cuda, dtype=DT[dtype]))
    for name, w in {**got, "state": left}.items():
        assert np.all((w >= 0) & (w <= 1 + 64 * U32 + U16)), name


@pytest.mark.parametrize("pattern", ["steps", "inside", "far inside", "blocks", "below", "years", "random"])
@pytest.mark.parametrize("dtype,hd", [("f32", 64), ("f32", 16), ("bf16", 64), ("bf16", 16)])
def test_decay_weights_where_timestamps_decrease(cuda, dtype, hd, pattern):
    """Two rows without a decrease between them weigh one another as defined, two
    on both sides of one by a number from 0 to 1, later rows not at all by earlier
    ones (exactly), and the other histories' bits do not change. A weight is a
    product of at most five factors and 1: 64 u32 of it, and a step of the output
    and the two-term operands in bf16 calls."""
    lengths, taus = (40, 200, 70), (0, 1, 60, 1)
    decay = (-0.01, -float(np.log(2.0)), -0.05, -0.01)
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    heads, T = R.DecayHeads(taus, decay, hd), int(cu[-1])
    rng = np.random.default_rng(3)
    others = torch.from_numpy(rng.standard_normal((T, 4 * hd))).to(cuda, DT[dtype])
    ts = np.concatenate([W.draw_timestamps(rng, n) for n in lengths])
    t = _times(pattern, 200).astype(np.int64)
    _, _, plain = _weights(cuda, dtype, hd, heads, cu, ts, 40, 240, others)
    ts[40:240] = 10 ** 9 + t
    got, left, rest = _weights(cuda, dtype, hd, heads, cu, ts, 40, 240, others)
    assert all(torch.equal(a, b) for a, b in zip(rest, plain))
    with pytest.raises(R.RestError) as e:
        R.decay_attn_forward(others, others, others, cu, heads, ts=torch.from_numpy(ts).to(cuda))
    assert e.value.status == 2
    drops = np.concatenate([[0], np.cumsum(np.diff(t) < 0)])
    i = np.arange(200)
    for h, (tau, g) in enumerate(zip(taus, decay)):
        n = i if tau == 0 else (t - t[0]) // tau
        known = (drops[:, None] == drops[None, :]) | (tau == 0)
        want = np.exp(np.minimum(g * (n[:, None] - n[None, :]), 0.0))
        tol = 64 * U32 + (U16 + 1.02 * 2 * 2.0 ** -16 if dtype == "bf16" else 0.0)
        low = i[:, None] >= i[None, :]
        for name, w in got.items():
            assert np.all(w[h][~low] == 0), (name, h)
            assert np.all(np.abs(w[h] - want)[low & known] <= tol * want[low & known] + 2.0 ** -120), (name, h)
            assert np.all((w[h][low] >= 0) & (w[h][low] <= 1 + tol)), (name, h)
        last = known[-1]
        assert np.all(np.abs(left[h] - want[-1])[last] <= 64 * U32 * want[-1][last] + 2.0 ** -120), h
        assert np.all((left[h] >= 0) & (left[h] <= 1 + 64 * U32)), h


# ---------------------------------------------------------------- streams


def _calls(cuda):
    """Every history call, with ``kw`` for the stream and what is given; by name."""
    torch.manual_seed(0)
    heads = R.DecayHeads((0, 64), (-0.1, -0.2), 32)
    x = [torch.randn(300, 64, device=cuda) for _ in range(4)]
    ts, cu = torch.arange(300, device=cuda) * 50, np.array([0, 300], dtype=np.int32)
    ids = torch.arange(300, device=cuda) % 40
    table = torch.randn(40, 64, device=cuda)

    def step(**kw):
        state = R.DecayState(heads, 300, device=cuda)
        torch.cuda.synchronize()
        return R.decay_attn_step(*x[:3], state, ts=ts, **kw)
    return {"embed_forward": lambda **kw: R.embed_forward(table, ids, **kw),
            "embed_backward": lambda **kw: R.embed_backward(x[0], ids, 40, **kw),
            "decay_attn_forward": lambda **kw: R.decay_attn_forward(*x[:3], cu, heads, ts=ts, **kw),
            "decay_attn_backward": lambda **kw: R.decay_attn_backward(*x, cu, heads, ts=ts, **kw),
            "decay_attn_step": step}


CALLS = ["embed_forward", "embed_backward", "decay_attn_forward", "decay_attn_backward", "decay_attn_step"]


@pytest.mark.parametrize("name", CALLS)
def test_a_call_allocates_on_its_stream(cuda, name, monkeypatch):
    """Outputs, workspace and status word of a call on another stream are that
    stream's memory: a block that the current stream has just freed may still be
    in use there."""
    call = _calls(cuda)[name]
    want = call()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    seen = []

    def watched(make):
        def made(*a, **kw):
            if str(kw.get("device", "")).startswith("cuda") or "like" in make.__name__:
                seen.append(torch.cuda.current_stream())
            return make(*a, **kw)
        return made

    torch.cuda.synchronize()
    with monkeypatch.context() as m:
        for f in ("empty", "empty_like", "zeros"):
            m.setattr(torch, f, watched(getattr(torch, f)))
        before = torch.cuda.current_stream()
        got = call(stream=other)
        assert torch.cuda.current_stream() == before
    if name == "decay_attn_step":
        seen = seen[4:]                       # the test's own state
    assert len(seen) >= 2 - (name == "decay_attn_step") and all(s == other for s in seen)
    torch.cuda.synchronize()
    for a, b in zip(got if isinstance(got, tuple) else (got,), want if isinstance(want, tuple) else (want,)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", CALLS)
def test_calls_without_the_stream_shortcut(cuda, name, monkeypatch):
    """torch's private names are a shortcut, not a need."""
    call = _calls(cuda)[name]
    want = call()
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert R._current_handle(torch.device("cuda", 0)) == side.cuda_stream
        got = call()
    torch.cuda.synchronize()
    for a, b in zip(got if isinstance(got, tuple) else (got,), want if isinstance(want, tuple) else (want,)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["embed_forward", "decay_attn_backward"])
def test_a_captured_call_does_not_read_its_status(cuda, name):
    """Refused whichever way the capturing stream is named, before anything is
    enqueued: the capture goes on, and replays what check=False put there."""
    call = _calls(cuda)[name]
    want = call()
    graph, side, calm = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side, capture_error_mode="thread_local"):
        with pytest.raises(ValueError, match="captured"):
            call()
        with torch.cuda.stream(calm):
            with pytest.raises(ValueError, match="captured"):
                call(stream=side)
        got = call(check=False)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got if isinstance(got, tuple) else (got,), want if isinstance(want, tuple) else (want,)):
        assert torch.equal(a, b)


def test_outputs_on_another_stream_outlive_their_use_on_the_current_one(cuda):
    """Memory of an output that the current stream still reads is not handed out again by its own stream."""
    calls = _calls(cuda)
    big = torch.randn(8192, 8192, device=cuda)
    want = calls["embed_forward"]()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    out = calls["embed_forward"](stream=other, check=False)
    torch.cuda.current_stream().wait_stream(other)
    for _ in range(4):
        big = big @ big                        # keeps the current stream busy
    kept = out.clone()
    where = out.data_ptr()
    del out
    again = calls["embed_forward"](stream=other, check=False)
    assert again.data_ptr() != where
    torch.cuda.synchronize()
    assert torch.equal(kept, want) and torch.equal(again, want)


# ---------------------------------------------------------------- states


def test_decay_state_takes_assigned_tensors(cuda):
    """A restored checkpoint, assigned as it is: the calls use it, and what it replaces stays as it was."""
    torch.manual_seed(2)
    heads = R.DecayHeads((0, 1), (-0.1, -0.2), 16)
    x, ts = torch.randn(2, 3, 32, device=cuda), [torch.tensor(t, device=cuda) for t in ([10, 20, 30], [15, 21, 40])]
    state = R.DecayState(heads, 3, device=cuda)
    R.decay_attn_step(x[0], x[0], x[0], state, ts=ts[0])
    saved = [t.clone() for t in (state.s, state.len, state.t_first, state.t_last)]
    want = R.decay_attn_step(x[1], x[1], x[1], state, ts=ts[1])
    old = [state.s, state.len, state.t_first, state.t_last]
    ended = [t.clone() for t in old]
    state.s, state.len, state.t_first, state.t_last = [t.clone() for t in saved]
    assert torch.equal(R.decay_attn_step(x[1], x[1], x[1], state, ts=ts[1]), want)
    assert all(torch.equal(a, b) for a, b in zip((state.s, state.len, state.t_first, state.t_last), ended))
    assert all(torch.equal(a, b) for a, b in zip(old, ended))
    state.s, state.len, state.t_first, state.t_last = [t.clone() for t in saved]
    o = R.decay_attn_forward(x[1], x[1], x[1], [0, 1, 2, 3], heads, ts=ts[1], state=state)
    # a one-row pass and the step: 12 u32 for each of the pass's products on the tensor pipe, and its weights'
    assert torch.all((o - want).abs() <= 200 * U32 * want.abs().max())
    assert all(torch.equal(a, b) for a, b in zip(old, ended))
    for name, bad in (("s", saved[0][:2]), ("s", saved[0].double()), ("len", saved[1].int()), ("t_last", saved[3].cpu())):
        with pytest.raises((TypeError, ValueError)):
            setattr(state, name, bad)
    assert state.s.shape == (3, 2, 16, 16)


def test_a_call_with_nothing_to_do_clears_the_status(cuda):
    """The word of an earlier call, whose error was not read, is not the empty call's."""
    heads = R.DecayHeads((0, 8), (-0.1, -0.1), 16)
    state = R.DecayState(heads, 2, device=cuda)
    x, i = torch.empty(0, 32, device=cuda), torch.empty(0, dtype=torch.int64, device=cuda)
    g = torch.zeros(4, 32, device=cuda)
    for call in (lambda **kw: R.embed_forward(g, i, **kw), lambda **kw: R.embed_backward(x, i, 4, **kw),
                 lambda **kw: R.embed_backward(x, i, 4, d_table=g, accumulate=True, **kw),
                 lambda **kw: R.decay_attn_forward(x, x, x, [0, 0], heads, ts=i, **kw),
                 lambda **kw: R.decay_attn_backward(x, x, x, x, [0, 0], heads, ts=i, **kw),
                 lambda **kw: R.decay_attn_step(x, x, x, state, ts=i, **kw)):
        err = torch.full((1,), 2, dtype=torch.int32, device=cuda)
        call(err=err, check=False)
        assert int(err) == 0
        err.fill_(2)
        call(err=err)


# ---------------------------------------------------------------- workspaces


def _launched(call):
    R.profile_begin()
    out = call()
    return out, {x["name"]: x["launches"] for x in R.profile_end()}


@pytest.mark.parametrize("dtype,hd,lengths", [("f32", 64, (1500,)), ("bf16", 32, (1500, 0, 700, 3)), ("f32", 16, (2000, 1000))])
def test_decay_in_a_smaller_workspace(cuda, dtype, hd, lengths):
    """The fastest cut's workspace, part of it, and the least: fewer segments, the
    same results within their bounds, nothing written behind the workspace."""
    (q, k, v, d_o), ts, cu, taus, decay = _case(dtype, hd, lengths, 3)
    heads = R.DecayHeads(taus, decay, hd)
    t, tts, L = [_dev(x, dtype) for x in (q, k, v, d_o)], torch.from_numpy(ts).to(cuda), max(lengths)
    want, S = O.decay_attention(q, k, v, ts, cu, taus, decay)
    mag, Smag = O.decay_attention(q, k, v, ts, cu, taus, decay, magnitude=True)
    ref = O.decay_attention_backward(q, k, v, ts, cu, taus, decay, d_o)
    big = O.decay_attention_backward(q, k, v, ts, cu, taus, decay, d_o, magnitude=True)
    full = R.decay_attn_workspace_size(R.REST_BF16 if dtype == "bf16" else R.REST_F32, heads, cu)
    least = R.decay_attn_workspace_size(R.REST_F32, heads, np.zeros(len(cu), dtype=np.int32))
    assert least < full
    seen = []
    for size in (full, full // 2 // 16 * 16, least):
        buf = torch.full((size + 4096,), 0xab, dtype=torch.uint8, device=cuda)
        ws = buf[:size]
        o, names = _launched(lambda: R.decay_attn_forward(*t[:3], cu, heads, ts=tts, ws=ws))
        state = R.DecayState(heads, len(lengths), device=cuda)
        o2 = R.decay_attn_forward(*t[:3], cu, heads, ts=tts, ws=ws, state=state)
        g, back = _launched(lambda: R.decay_attn_backward(*t, cu, heads, ts=tts, ws=ws))
        assert bool((buf[size:] == 0xab).all())
        for a, b, m, what in ((o, want, mag, "o"), (o2, want, mag, "o with a state"), *zip(g, ref, big, ("dq", "dk", "dv"))):
            if dtype == "bf16":
                _rounded_once(a, b, m, L, hd, what)
            else:
                err = np.abs(a.cpu().numpy().astype(np.float64) - b)
                assert np.all(err <= (L + 2 * hd + 64) * U32 * m), what
        assert np.all(np.abs(state.s.cpu().numpy() - S) <= (L + 64) * U32 * Smag)
        seen.append(("decay_parts" in names, "decay_parts" in back))
    assert seen[0] == (True, True) and seen[-1] == (False, False)
    with pytest.raises(R.RestError) as e:
        R.decay_attn_forward(*t[:3], cu, heads, ts=tts, ws=torch.empty(least - 256, dtype=torch.uint8, device=cuda))
    assert e.value.status == 6


@pytest.mark.parametrize("dtype,hd,lengths", [("bf16", 32, (300,) * 90), ("f32", 32, (300,) * 90), ("bf16", 64, (200, 330) * 20)])
def test_decay_histories_that_are_not_cut(cuda, dtype, hd, lengths):
    """The histories that other tests take for uncut ones: the pass alone is launched."""
    taus, decay = (0, 0, 0, 0, 1, 64, 4096, 65536), (-0.1, -0.01, -0.5, 0.0, -1e-5, -1e-3, -0.02, -0.3)
    (q, k, v, d_o), ts, cu, taus, decay = _case(dtype, hd, lengths, 31, taus=taus, decay=decay)
    heads = R.DecayHeads(taus, decay, hd)
    t, tts = [_dev(x, dtype) for x in (q, k, v, d_o)], torch.from_numpy(ts).to(cuda)
    _, names = _launched(lambda: R.decay_attn_forward(*t[:3], cu, heads, ts=tts))
    assert set(names) - {"decay_prep"} == {"decay_pass"}
    _, names = _launched(lambda: R.decay_attn_backward(*t, cu, heads, ts=tts))
    assert set(names) - {"decay_prep"} == {"decay_pass", "decay_dkdv"}


# ---------------------------------------------------------------- threads


def test_decay_calls_from_several_threads(cuda):
    """Batches whose launches take different amounts of shared memory, each from a
    thread and stream of its own: no call refused, the same bits as alone."""
    heads = R.DecayHeads((0, 0, 0, 0), (-0.1, -0.01, -0.3, 0.0), 64)
    torch.manual_seed(4)
    cases = []
    for lengths in ((64,), (300,) * 10, (64,) * 148, (640,) * 3, (70,) * 300, (5000,)):
        cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
        x = [torch.randn(int(cu[-1]), 256, device=cuda).bfloat16() for _ in range(4)]
        cases.append((cu, x, R.decay_attn_forward(*x[:3], cu, heads), R.decay_attn_backward(*x, cu, heads)))
    torch.cuda.synchronize()
    wrong = []

    def work(cu, x, o, grads):
        try:
            stream = torch.cuda.Stream()
            for _ in range(40):
                got = R.decay_attn_forward(*x[:3], cu, heads, stream=stream)
                back = R.decay_attn_backward(*x, cu, heads, stream=stream)
                stream.synchronize()
                if not torch.equal(got, o) or not all(torch.equal(a, b) for a, b in zip(back, grads)):
                    wrong.append("other bits")
        except Exception as e:  # noqa: BLE001
            wrong.append(repr(e))

    threads = [threading.Thread(target=work, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:3]


# ---------------------------------------------------------------- waits that run out


def _step_case(cuda, dtype, hd, H, n):
    torch.manual_seed(n)
    heads = R.DecayHeads(([0, 64] * 16)[:H], [-0.1] * H, hd)
    state = R.DecayState(heads, n + 1, device=cuda)
    state.s.normal_()
    state.len.fill_(3)
    state.t_first.fill_(1000)
    state.t_last.fill_(2000)
    x = [torch.randn(n, H * hd, device=cuda).to(DT[dtype]) for _ in range(3)]
    slots = torch.randperm(n + 1, device=cuda)[:n].int()
    return x, state, torch.full((n,), 2500, device=cuda), slots


@pytest.mark.parametrize("dtype,hd,H,n", [("bf16", 64, 8, 3), ("f32", 16, 2, 1), ("bf16", 32, 32, 40), ("f32", 64, 8, 700)])
def test_a_step_whose_waits_run_out_leaves_its_state(cuda, dtype, hd, H, n):
    """One block and several to an entry, one chunk and several to a block: nothing
    of a chunk that did not arrive is stored, no token is counted, and the next
    call is right."""
    x, state, ts, slots = _step_case(cuda, dtype, hd, H, n)
    kept = [t.clone() for t in (state.s, state.len, state.t_first, state.t_last)]
    o = torch.full_like(x[0], 7.0)
    assert R.selftest_decay_step_timeout(*x, state, o, ts=ts, slots=slots) == 5
    assert all(torch.equal(a, b) for a, b in zip((state.s, state.len, state.t_first, state.t_last), kept))
    assert torch.all(o == 7.0)
    fresh = R.DecayState(state.heads, n + 1, tensors=kept)
    want = R.decay_attn_step(*x, fresh, ts=ts, slots=slots)
    assert torch.equal(R.decay_attn_step(*x, state, ts=ts, slots=slots), want)
    assert torch.equal(state.s, fresh.s) and torch.equal(state.len, fresh.len)


def test_a_timeout_is_reported_over_a_bad_slot(cuda):
    """The bad slot's entry reports at once, the others' waits run out later: the
    code that voids their outputs is the one that is left."""
    x, state, ts, slots = _step_case(cuda, "bf16", 32, 8, 20)
    slots[3] = 99
    o = torch.full_like(x[0], 7.0)
    assert R.selftest_decay_step_timeout(*x, state, o, ts=ts, slots=slots) == 5
    with pytest.raises(R.RestError) as e:
        R.decay_attn_step(*x, state, ts=ts, slots=slots)
    assert e.value.status == 1


# ---------------------------------------------------------------- tiles that are filled again


@pytest.mark.parametrize("hd", [16, 32, 64])
def test_decay_gradients_of_ragged_ends_repeat(cuda, hd):
    """Uncut histories of six blocks, the last of 13 rows: the backward pass starts
    there, with zeros written into tiles that are filled again three blocks on.
    Equal calls give equal bits, and each history's are those of its own batch."""
    torch.manual_seed(hd)
    H, n, L = 8, 90, 333
    heads = R.DecayHeads((0,) * H, (-0.01,) * H, hd)
    x = [torch.randn(n * L, H * hd, device=cuda).bfloat16() for _ in range(4)]
    cu = np.arange(n + 1, dtype=np.int32) * L
    least = torch.empty(R.decay_attn_workspace_size(R.REST_BF16, heads, [0] * (n + 1)), dtype=torch.uint8, device=cuda)
    want = R.decay_attn_backward(*x, cu, heads, ws=least)
    one = R.decay_attn_backward(*(t[:L] for t in x), cu[:2], heads, ws=least[:R.decay_attn_workspace_size(1, heads, [0, 0])])
    assert all(torch.equal(a[:L], b) for a, b in zip(want, one))
    for _ in range(50):
        assert all(torch.equal(a, b) for a, b in zip(R.decay_attn_backward(*x, cu, heads, ws=least), want))
