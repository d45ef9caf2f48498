"""The 4-bit key-value cache where its operators are easily wrong: zero rows and zero keys, lengths and
rows beyond what a table or a tensor holds, groups of different magnitude, weights far below the
largest, replays of captured graphs.  Tolerances as in test_kv4.py, plus what stands at a test.
"""
import subprocess

import numpy as np
import pytest
import torch

import kv4_plain as KP
from test_kv4 import DT, Batch, _check, _fast_fill, _rows, _status, _tolerance, kv4  # noqa: F401


def _token(b, seq, pos, side, head):
    """The levels' bytes and the pairs (uint16 [d / 32, 2]: scale, low) of one key (side 0) or value of the
    host's cache, as views."""
    off, d = pos % b.page, b.d
    rec = b.cache[b.table[seq, pos // b.page], head, side].reshape(-1)
    at = b.page * d // 2 + off * d // 8
    return rec[off * d // 2:(off + 1) * d // 2], rec[at:at + d // 8].view(np.uint16).reshape(-1, 2)


def _constant(b, seq, pos, side, value):
    """The key or value of a token at all heads: constant groups of a value that bf16 holds."""
    bits = np.float32(value).view(np.uint32)
    assert bits & 0xFFFF == 0
    for h in range(b.hkv):
        levels, pairs = _token(b, seq, pos, side, h)
        levels[:], pairs[:, 0], pairs[:, 1] = 0, 0, bits >> 16


# -------------------------------------------------------------------------- zero rows, zero and huge keys

@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 33, 49, 300])
def test_zero_rows_and_zero_keys(kv4, cuda, d, new):
    """A chunk of zeros over zero keys, zeros behind a prompt (a tile of 128 and more), zero rows over keys
    and rows over zero keys: few rows, and many with one and with two query tiles."""
    rng = np.random.default_rng(new + d)
    lens = [new, 700, 400, 450]
    b = _fast_fill(Batch(lens, [min(new, n) for n in lens], 32, 2, d, seed=new), rng)
    for s, first in ((0, 0), (1, 250), (3, 0)):
        for pos in range(first, lens[s]):
            _constant(b, s, pos, 0, 0.0)
    b.gpu()
    q = _rows(rng, 2, b.total, d, "bf16", True, 1.5)
    q[:, :b.cu[3]] = 0
    out = torch.full_like(q, 3.0)
    kv4.attend(b.g_cache, q, *b.g, new, out=out)
    assert _status(kv4) == 0
    _check(kv4, b, q, out, out)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 33, 300])
def test_a_dry_run_of_zeros(kv4, cuda, d, new):
    """Zeros over a cache of zeros are zeros; rows before the first token too, which are reported."""
    cache = kv4.empty(12, 2, 64, d)
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(2, 6)
    q = torch.zeros(8, 2 * new, d, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, new, 2 * new], dtype=torch.int32, device="cuda")
    for short, status in ((new, 0), (new // 2, 6)):
        lens = torch.tensor([300, short], dtype=torch.int32, device="cuda")
        out = torch.full_like(q, 3.0)
        kv4.attend(cache, q, table, lens, cu, new, out=out)
        assert _status(kv4) == status and (out == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [2, 33, 300])
def test_zero_rows_over_pages_outside_the_cache(kv4, cuda, d, new):
    """A tile of tokens whose pages all lie outside the cache: a zero row's weights are equal over the others."""
    rng = np.random.default_rng(new)
    n = 128 * 3 + new
    b = _fast_fill(Batch([n], [new], 32, 1, d, seed=2), rng).gpu()
    b.g[0][0, 4:8] = torch.tensor([b.pages, -1, b.pages + 9, -7], dtype=torch.int32, device="cuda")
    q = torch.zeros(2, new, d, dtype=torch.bfloat16, device="cuda")
    out = kv4.attend(b.g_cache, q, *b.g, new).double().cpu().numpy()
    assert _status(kv4) == 6
    v = KP.tokens(KP.decode(b.cache), b.table[0], n)[1][:, 0].astype(np.float64)
    v[128:256] = 0
    want = np.cumsum(v, 0)[n - new:] / (np.arange(n - new, n) + 1 - 128)[:, None]
    assert (np.abs(out - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * np.abs(v).max()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_keys_near_the_end_of_the_range(kv4, cuda, d):
    """Keys up to 2^121 against rows of 2^-122: ordinary logits (all of it powers of two, so exact)."""
    rng = np.random.default_rng(d)
    new, n = 70, 300
    b = _fast_fill(Batch([n], [new], 32, 1, d, seed=3), rng)
    for pos in range(n):
        _constant(b, 0, pos, 0, float(rng.choice([-1, 1])) * 2.0 ** int(rng.integers(119, 122)))
    b.gpu()
    sign = torch.from_numpy(rng.choice([-1.0, 1.0], (2, new, 1))).cuda()
    q = (sign * 2.0 ** -122).expand(2, new, d).to(torch.bfloat16).contiguous()
    out = kv4.attend(b.g_cache, q, *b.g, new)
    assert _status(kv4) == 0
    _check(kv4, b, q, out, out)


@pytest.mark.gpu
@pytest.mark.parametrize("new,dtype", [(1, "bf16"), (1, "fp32"), (3, "bf16"), (3, "fp32"), (70, "bf16")])
def test_zero_rows_at_a_tiny_logit_scale(kv4, cuda, new, dtype):
    """Weights are equal then, for zero rows and for others."""
    rng = np.random.default_rng(new)
    b = _fast_fill(Batch([77 + new, 200], [new, new], 32, 2, 64, seed=6), rng).gpu()
    q = _rows(rng, 4, b.total, 64, dtype, True)
    q[:, ::2] = 0
    for scale in (1e-30, 1e-38):
        out = kv4.attend(b.g_cache, q, *b.g, new, sm_scale=scale)
        assert _status(kv4) == 0
        _check(kv4, b, q, out, out, scale=float(np.float32(scale)), dtype=dtype)


# ---------------------------------------------------------------- lengths and rows beyond what is there

@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,over", [(1, 1), (4, 3), (4, 6), (70, 9)])
def test_a_length_beyond_the_table(kv4, cuda, d, new, over):
    """The rows whose tokens the table cannot name are skipped and reported; the others are the tokens that
    they are, and no other token of the cache is touched."""
    rng = np.random.default_rng(new + over)
    page, hkv, hq, n = 16, 2, 4, 160
    b = _fast_fill(Batch([n, 45], [new, min(new, 45)], page, hkv, d, seed=4), rng).gpu()
    table = b.g[0][:, :n // page].contiguous()
    lens = b.g[1].clone()
    lens[0] = n + over
    have = max(0, new - over)                                        # rows of sequence 0 with a place
    k, v = (_rows(rng, hkv, b.total, d, "bf16", True) for _ in range(2))
    ks, vs = (torch.full((hkv, b.total, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kv4.append(b.g_cache, k, v, table, lens, b.g[2], k_stored=ks, v_stored=vs)
    assert _status(kv4) == 6
    xk, xv = k.float().cpu().numpy(), v.float().cpu().numpy()
    for t in range(have):
        b.put(0, n + over - new + t, xk[:, t], xv[:, t])
    for t in range(new, b.total):
        b.put(1, 45 - b.total + t, xk[:, t], xv[:, t])
    assert np.array_equal(b.g_cache.cpu().numpy(), b.cache)
    assert (ks[:, have:new] == 9).all() and (vs[:, have:new] == 9).all()
    ko, vo = (torch.full_like(ks, 9.0) for _ in range(2))
    kv4.read(b.g_cache, table, lens, b.g[2], k_out=ko, v_out=vo)
    assert _status(kv4) == 6
    for got, want in ((ko, ks), (vo, vs)):
        assert (got[:, have:new] == 0).all()
        assert torch.equal(got[:, :have], want[:, :have]) and torch.equal(got[:, new:], want[:, new:])
    q = _rows(rng, hq, b.total, d, "bf16", True, 1.5)
    out = torch.full_like(q, 3.0)
    kv4.attend(b.g_cache, q, table, lens, b.g[2], new, out=out)
    assert _status(kv4) == 6 and (out[:, have:new] == 0).all()
    decoded = KP.decode(b.cache)
    for s, rows, at in ((0, range(have), n + over - new), (1, range(new, b.total), 45 - b.total)):
        for t in rows:                                                # one row at a time: its tokens end at its own
            pos = at + t
            want, size, span = KP.attend(decoded, q[:, t:t + 1].float().cpu().numpy(), b.table[s:s + 1],
                                         [pos + 1], np.array([0, 1]))
            err = np.abs(out[:, t:t + 1].float().cpu().numpy() - want)
            assert (err <= _tolerance(want, size, span, "bf16", n, d)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("new", [5, 70])
@pytest.mark.parametrize("first,last", [(0, 2), (0, "new"), (-2, 0), (-2, 3)])
def test_rows_that_the_tensors_do_not_have(kv4, cuda, new, first, last):
    """cu_new names rows before the tensors' first or behind their last: the rows that are there are the tokens
    that cu_new says, in all three operators, and the rest is reported."""
    rng = np.random.default_rng(new + 10)
    page, d, hkv, hq = 32, 64, 2, 4
    b = _fast_fill(Batch([300, 90], [new, new], page, hkv, d, seed=7), rng).gpu()
    lo, hi = -first, b.total - (new + 2 if last == "new" else last)      # rows of the whole batch that are there
    cu = b.g[2] + first
    k, v = (_rows(rng, hkv, b.total, d, "bf16", True) for _ in range(2))
    kv4.append(b.g_cache, k[:, lo:hi], v[:, lo:hi], *b.g[:2], cu)
    assert _status(kv4) == 6
    xk, xv = k.float().cpu().numpy(), v.float().cpu().numpy()
    for t in range(lo, hi):
        s = int(t >= new)
        b.put(s, b.lens[s] - b.cu[s + 1] + t, xk[:, t], xv[:, t])
    assert np.array_equal(b.g_cache.cpu().numpy(), b.cache)
    ko = torch.full((hkv, hi - lo, d), 9.0, dtype=torch.float32, device="cuda")
    kv4.read(b.g_cache, *b.g[:2], cu, k_out=ko)
    assert _status(kv4) == 6
    decoded = KP.decode(b.cache)
    for t in range(lo, hi):
        s = int(t >= new)
        pos = b.lens[s] - b.cu[s + 1] + t
        assert np.array_equal(ko[:, t - lo].cpu().numpy(), KP.tokens(decoded, b.table[s], b.lens[s])[0][pos])
    q = _rows(rng, hq, b.total, d, "bf16", True, 1.5)
    out = torch.full((hi - lo, hq, d), 3.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    kv4.attend(b.g_cache, q[:, lo:hi], *b.g[:2], cu, new, out=out)
    assert _status(kv4) == 6
    want, size, span = KP.attend(decoded, q.float().cpu().numpy(), b.table, b.lens, b.cu)
    err = np.abs(out.float().cpu().numpy() - want[:, lo:hi])
    assert (err <= _tolerance(want, size, span, "bf16", 300, d)[:, lo:hi]).all()


# ------------------------------------------------------------------------- groups and weights far apart

def _spans(b, hq, seq=0):
    """[Hq, T, d / 32]: the largest |value| of each group that a row sees, and [Hq, 1, d / 32] the largest scale."""
    n, new = b.lens[seq], b.new[seq]
    v = np.abs(KP.tokens(KP.decode(b.cache), b.table[seq], n)[1])            # [n, Hkv, d]
    most = np.maximum.accumulate(v.reshape(n, b.hkv, -1, 32).max(-1), 0)[n - new:]
    scale = np.stack([[(_token(b, seq, pos, 1, h)[1][:, 0].astype(np.uint32) << 16).view(np.float32)
                       for h in range(b.hkv)] for pos in range(n)]).max(0)
    share = hq // b.hkv
    return most.transpose(1, 0, 2).repeat(share, 0).astype(np.float64), scale[:, None].repeat(share, 0).astype(np.float64)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 16, 70])
def test_groups_of_different_magnitude(kv4, cuda, d, new):
    """Values whose groups differ by 2^11 (few rows) and 2^24 (many): each group to its own precision, 2^-11 of
    its largest value for the weights and as much for the values.  Beside that, few rows: a weight times a
    scale is rounded to 2^-31 of the largest value's magnitude at least, and multiplies at most 8; many rows: a
    value to 2^-15 of its group's largest scale."""
    rng = np.random.default_rng(new + d)
    n, hkv, hq = 300 + new, 1, 2
    many = new * hq > 48
    b = _fast_fill(Batch([n], [new], 32, hkv, d, seed=5), rng)
    power = np.array([0, -20, 4, -9] if many else [0, -10, 1, -5])[:d // 32]
    for pos in range(n):
        p = _token(b, 0, pos, 1, 0)[1]
        f = (p.astype(np.uint32) << 16).view(np.float32) * (2.0 ** (power + rng.integers(-1, 2)))[:, None].astype(np.float32)
        p[:] = f.view(np.uint32) >> 16
    b.gpu()
    q = _rows(rng, hq, new, d, "bf16", True, 1.2)
    out = kv4.attend(b.g_cache, q, *b.g, new)
    assert _status(kv4) == 0
    want, size, _ = KP.attend(KP.decode(b.cache), q.float().cpu().numpy(), b.table, b.lens, b.cu)
    span, scale = _spans(b, hq)
    floor = 2.0 ** -15 * scale if many else n * 8 * 2.0 ** -31 * span.max() * np.ones_like(scale)
    tol = (2.0 ** -11 * span * (2 + 2 * size) + floor).repeat(32, -1) + 2.0 ** -8 * np.abs(want)
    err = np.abs(out.float().cpu().numpy() - want)
    assert (err <= tol).all(), ((err / tol).reshape(hq, new, -1, 32).max((0, 1, 3)))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [70, 300])
def test_weights_far_below_the_largest(kv4, cuda, d, new):
    """Many rows: a token that takes nearly all of the weight and whose value is 0, before 4096 tokens of 2^-22.7
    of its weight each, so that the output is theirs; in 148 sequences on the same pages, so that each is
    about one CTA's.  Keys are constant groups: the logits are exact but for their own roundings in the
    exponentials' arguments (2^-24 of 23, twice).  A weight is kept to half a step of fp16 denormals beside a
    largest one of 2^7, so to 2^-25 of 2^-15.7; a value to 2^-11 of it and 2^-15 of its scale."""
    others, seqs = 4096, 148
    top = {128: 1.390625, 64: 1.96875}[d]                    # sqrt(d) * top * log2(e) = 22.7
    n = 1 + others + new
    rng = np.random.default_rng(new)
    b = _fast_fill(Batch([n], [new], 128, 1, d, seed=9), rng)
    rec = b.cache.reshape(b.pages, 1, 2, -1)
    rec[:, :, 0] = 0
    pair = np.array([1.0 / 16, 1.0], np.float32).view(np.uint32) >> 16
    rec[:, :, 1, b.page * d // 2:] = np.tile(pair.astype(np.uint16).view(np.uint8), (b.pages, 1, b.page * d // 32))
    _constant(b, 0, 0, 0, top)
    _constant(b, 0, 0, 1, 0.0)
    b.gpu()
    table, lens = b.g[0].repeat(seqs, 1), b.g[1].repeat(seqs)
    cu = torch.arange(seqs + 1, dtype=torch.int32, device="cuda") * new
    q = torch.ones(1, seqs * new, d, dtype=torch.bfloat16, device="cuda")
    out = kv4.attend(b.g_cache, q, table, lens, cu, new)
    assert _status(kv4) == 0
    want = KP.attend(KP.decode(b.cache), q[:, :new].float().cpu().numpy(), b.table, b.lens, b.cu)[0]
    err = np.abs(out.float().cpu().numpy().reshape(seqs, new, d) - want)
    rel = 2.0 ** -8 + 2.0 ** -9.3 + 2.0 ** -11 + 2.0 ** -15 + 2.0 ** -18
    assert (err <= rel * np.abs(want)).all(), (err / np.abs(want)).max()


# ------------------------------------------------------------------------------ captured and replayed

@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d,new", [(8, 2, 128, 70), (4, 2, 64, 150), (8, 2, 64, 3)])
def test_replays_share_out_the_tokens_anew(kv4, cuda, hq, hkv, d, new):
    """Two graphs on one workspace, with append and the attention of many rows (and of few), replayed in turn with
    other lengths and numbers of rows: contexts that all CTAs share, that some share, that none shares, and
    sequences without a row; also on a stream of its own, and with other memory in the workspace between."""
    rng = np.random.default_rng(new)
    page, most = 64, 5000
    b = _fast_fill(Batch([most, most], [new, new], page, hkv, d, seed=8), rng).gpu()
    k, v = (_rows(rng, hkv, b.total, d, "bf16", True) for _ in range(2))
    q = _rows(rng, hq, b.total, d, "bf16", True, 1.5)
    p = kv4.Params(hq, hkv, d, page, b.pages, b.table.shape[1], 2, b.total, new, 0)
    size = kv4.attend_workspace_bytes(p)
    assert size > 0
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(q) for _ in range(2)]
    kv4.append(b.g_cache, k, v, *b.g)
    kv4.attend(b.g_cache, q, *b.g, new, out=outs[0], workspace=ws)
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kv4.append(b.g_cache, k, v, *b.g)
            kv4.attend(b.g_cache, q, *b.g, new, out=o, workspace=ws)
        graphs.append(g)
    side = torch.cuda.Stream()
    for step, (lens, rows) in enumerate((([most, 700], [new, new]), ([new, 1], [new, 1]), ([3000, 129], [0, 1]),
                                         ([most, most], [new, 2]), ([128, 77], [min(new, 128), 1]),
                                         ([1411, 3001], [new // 2, new]))):
        b.lens, b.new, b.cu = lens, rows, np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        b.g[1].copy_(torch.tensor(lens, dtype=torch.int32))
        b.g[2].copy_(torch.from_numpy(b.cu))
        for x, heads in ((q, hq), (k, hkv), (v, hkv)):
            x.copy_(_rows(rng, heads, b.total, d, "bf16", True, 1.5))
        ws.fill_(step * 51)
        for o in outs:
            o.fill_(3.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(side if step % 2 else torch.cuda.current_stream()):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        xk, xv = k.float().cpu().numpy(), v.float().cpu().numpy()
        for s, n in enumerate(lens):
            for t in range(b.cu[s], b.cu[s + 1]):
                b.put(s, n - b.cu[s + 1] + t, xk[:, t], xv[:, t])
        assert _status(kv4) == 0
        for o in outs:
            _check(kv4, b, q, o, torch.full_like(q, 3.0))
    del graphs


# ------------------------------------------------------- CPU: the words that hand over partial results

READY = r'''
#include <cstdint>
#include <cstdio>
#include <functional>
#include "kv4_ready.h"
using namespace sbsa;
// One word, and what the other side does between two accesses of this side (once).
struct Word {
  uint64_t* at;
  std::function<void()>* between;
  void step() const {
    if (between && *between) {
      auto f = *between;
      *between = nullptr;
      f();
    }
  }
  uint64_t load() const { return *at; }
  uint64_t exchange(uint64_t x) const {
    const uint64_t old = *at;
    *at = x;
    step();
    return old;
  }
  void store(uint64_t x) const { *at = x; }
};
int main() {
  const uint64_t call = 0x123456789ABCDEF1ull, other = 0x0F0F0F0F0F0F0F05ull;
  int bad = 0;
  auto is = [&](bool good, const char* what, int order, int failed) {
    if (!good) ++bad, printf("%s: order %d, failed %d\n", what, order, failed);
  };
  const uint64_t held[] = {0, other, other + 1, other + 2, ~(uint64_t)0, call + 4};
  for (uint64_t before : held)
    for (int failed = 0; failed < 2; ++failed) {
      uint64_t word = before;
      const Word w{&word, nullptr};
      // an ordinary call: nothing there, then there, then cleared
      is(ready_look(w, call) == kReadyNot, "nothing yet", 0, failed);
      ready_publish(w, call, failed != 0);
      is(ready_look(w, call) == (failed ? kReadyFailed : kReadyPart), "published", 0, failed);
      ready_leave(w, call, false);
      is(word == 0, "left as 0", 0, failed);
      // a joiner that gives up, before, after and in the middle of publishing: no later run of the same
      // call (a replay) may find a part, nor a joiner that has gone
      for (int order = 0; order < 4; ++order) {
        word = before;
        std::function<void()> none, leave = [&] { ready_leave(Word{&word, nullptr}, call, true); },
                              publish = [&] { ready_publish(Word{&word, nullptr}, call, failed != 0); };
        if (order == 0) publish(), leave();
        if (order == 1) leave(), publish();
        if (order == 2) ready_publish(Word{&word, &leave}, call, failed != 0);
        if (order == 3) ready_leave(Word{&word, &publish}, call, true);
        is(ready_look(w, call) == kReadyNot, "after giving up", order, failed);
        ready_publish(w, call, false);
        is(ready_look(w, call) == kReadyPart, "the next run", order, failed);
        ready_leave(w, call, false);
        is(word == 0, "the next run's end", order, failed);
      }
    }
  return bad != 0;
}
'''


def test_words_of_shared_items_are_clean_after_a_failure(tmp_path):
    """A partial result's word, in every order of the CTA that leaves the part and the one that takes it or
    gives up: afterwards it holds nothing that the same call, replayed in a graph, would take for a part."""
    import block_sparse_attention_sbsa_b200.build as build
    src, exe = tmp_path / "ready.cpp", tmp_path / "ready"
    src.write_text(READY)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", build.CSRC, "-o", str(exe), str(src)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
