"""The 4-bit key-value cache: append and read bit for bit against a plain
numpy form of the format, attention against float64 on what the cache stands
for, at the sizes, masks, orders and strides where it can go wrong; refusals
on the CPU.

Tolerances of attention.  With rows' true output o, let |V| be the largest
cached value a row sees and Z the largest |q| . |k| * scale over its tokens.
bf16: the output's rounding, 2^-8 |o|; every weight is rounded to fp16 before
its product with a value, at most 2^-11 of it, so at most 2^-11 |V|; a kernel
may take the cached values in fp16, 2^-11 of each: of a value at most 2^-11 |V|,
of a key at most 2^-11 Z in a logit, which moves each weight by that much of itself and
its sum too, 2 * 2^-11 Z |V|.  fp32: the sums of a logit in fp32 in any order, and
the two-part products' 2^-22, at most (d + 16) 2^-23 Z in the worst case, doubled
as above; exponentials to 2^-21 with their argument's rounding 2^-23 * 2 Z; the sums
over n tokens, taken in parts, 2^-23 * (64 + n / 64).
"""
import ctypes

import numpy as np
import pytest
import torch

import kv4_plain as KP

FAKE = ctypes.c_void_p(1 << 20)   # aligned, never dereferenced on the host
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def kv4():
    from block_sparse_attention_sbsa_b200 import build
    build.build()
    from block_sparse_attention_sbsa_b200 import kv4
    return kv4


# ------------------------------------------------------------------------------------ CPU: refusals

def _params(kv4, **kw):
    base = dict(n_q_heads=8, n_kv_heads=2, head_dim=128, page_size=64, n_pages=10, max_pages=5,
                n_seqs=2, n_tokens=3, max_new=2, dtype=0, list_heads=0, block_size=0,
                max_blocks=0, sm_scale=0.0)
    base.update(kw)
    return kv4.Params(**base)


def _append(kv4, p, cache=FAKE, k=FAKE, v=FAKE, strides=(256, 128, 256, 128), stored=None, table=FAKE):
    return kv4.lib.sbsa_kv4_append(ctypes.byref(p), cache, table, FAKE, FAKE, k, strides[0], strides[1],
                                   v, strides[2], strides[3], stored, None, None)


def _read(kv4, p, cache=FAKE, out=FAKE, lens=FAKE):
    return kv4.lib.sbsa_kv4_read(ctypes.byref(p), cache, FAKE, lens, FAKE, out, None, None)


def _attend(kv4, p, q=FAKE, o=FAKE, strides=(1024, 128, 1024, 128), idx=None, cnt=None, ws=FAKE,
            ws_bytes=1 << 30):
    return kv4.lib.sbsa_kv4_attend(ctypes.byref(p), FAKE, FAKE, FAKE, FAKE, q, strides[0], strides[1],
                                   o, strides[2], strides[3], idx, cnt, ws, ws_bytes, None)


def _all(kv4, p):
    return _append(kv4, p), _read(kv4, p), _attend(kv4, p)


@pytest.mark.parametrize("change,code", [
    (dict(n_kv_heads=0), 1), (dict(n_pages=0), 1), (dict(max_pages=0), 1), (dict(n_seqs=-1), 1),
    (dict(n_tokens=-1), 1), (dict(dtype=2), 1), (dict(head_dim=0), 1), (dict(head_dim=96), 2),
    (dict(page_size=0), 1), (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=256), 2),
    (dict(max_pages=1 << 25, page_size=64), 2), (dict(n_kv_heads=65536, n_q_heads=65536), 2),
])
def test_every_operator_refuses(kv4, change, code):
    p = _params(kv4, **change)
    assert _all(kv4, p) == (code,) * 3
    assert kv4.lib.sbsa_kv4_cache_bytes(ctypes.byref(p)) == 0
    assert kv4.lib.sbsa_kv4_attend_workspace_bytes(ctypes.byref(p)) == 0


@pytest.mark.parametrize("change,code", [
    (dict(n_q_heads=7), 1), (dict(n_q_heads=0), 1), (dict(max_new=0), 1), (dict(sm_scale=-1.0), 1),
    (dict(sm_scale=float("nan")), 1), (dict(sm_scale=float("inf")), 1),
    (dict(list_heads=4, block_size=64, max_blocks=1), 1),          # neither Hkv nor Hq
    (dict(list_heads=2, block_size=64, max_blocks=0), 1), (dict(list_heads=2, block_size=0, max_blocks=1), 1),
    (dict(list_heads=2, block_size=32, max_blocks=1), 2),
    (dict(list_heads=2, block_size=64, max_blocks=1, page_size=128), 1),   # half a page
    (dict(list_heads=2, block_size=128, max_blocks=1 << 24), 2),
    (dict(n_tokens=1 << 29), 2), (dict(n_seqs=1 << 29), 2),
])
def test_attend_refuses(kv4, change, code):
    p = _params(kv4, **change)
    lists = FAKE if p.list_heads else None
    assert _attend(kv4, p, idx=lists, cnt=lists) == code


def test_pointers_strides_and_workspace_are_checked(kv4):
    p = _params(kv4)
    odd = ctypes.c_void_p((1 << 20) + 8)
    assert _append(kv4, p, cache=None) == 1 and _append(kv4, p, k=None) == 1 and _append(kv4, p, v=None) == 1
    assert _append(kv4, p, table=None) == 1 and _append(kv4, p, cache=odd) == 1 and _append(kv4, p, k=odd) == 1
    assert _append(kv4, p, stored=odd) == 1
    for i in range(4):
        for bad in (-128, 132):
            s = [256, 128, 256, 128]
            s[i] = bad
            assert _append(kv4, p, strides=s) == 1 and _attend(kv4, p, strides=s) == 1
    f32 = _params(kv4, dtype=1)
    assert _append(kv4, f32, strides=(256, 130, 256, 128)) == 1
    assert _read(kv4, p, cache=None) == 1 and _read(kv4, p, out=odd) == 1 and _read(kv4, p, lens=None) == 1
    assert _attend(kv4, p, q=None) == 1 and _attend(kv4, p, o=odd) == 1
    assert _attend(kv4, p, idx=FAKE, cnt=FAKE) == 1                     # lists without list_heads
    lists = _params(kv4, list_heads=2, block_size=64, max_blocks=3)
    assert _attend(kv4, lists, idx=FAKE) == 1 and _attend(kv4, lists) == 1
    need = kv4.attend_workspace_bytes(p)
    assert need > 0
    assert _attend(kv4, p, ws=None) == 3 and _attend(kv4, p, ws_bytes=need - 1) == 3
    assert _attend(kv4, p, ws=ctypes.c_void_p((1 << 20) + 128)) == 3
    null = kv4.lib.sbsa_kv4_append(None, *[FAKE] * 5, 0, 0, FAKE, 0, 0, None, None, None)
    assert null == 1


def test_nothing_to_do_enqueues_nothing(kv4):
    for change in (dict(n_seqs=0), dict(n_tokens=0)):
        p = _params(kv4, **change)
        assert _append(kv4, p, cache=None, k=None, v=None) == 0
        assert _read(kv4, p, cache=None, out=None) == 0
        assert _attend(kv4, p, q=None, o=None, ws=None, ws_bytes=0) == 0


def test_workspace_is_needed_where_tokens_can_be_shared_out(kv4):
    for change, none in ((dict(max_pages=2), True), (dict(max_pages=3), False),
                         (dict(max_pages=2, max_new=13), False),              # 52 rows of a kv head
                         (dict(list_heads=2, block_size=64, max_blocks=2), True),
                         (dict(list_heads=2, block_size=64, max_blocks=3), False)):
        assert (kv4.attend_workspace_bytes(_params(kv4, **change)) == 0) == none


def test_cache_bytes_and_params_layout(kv4):
    p = _params(kv4)
    assert kv4.lib.sbsa_kv4_cache_bytes(ctypes.byref(p)) == 10 * 2 * 2 * 64 * 80
    assert ctypes.sizeof(kv4.Params) == 14 * 4 and kv4.Params.sm_scale.offset == 13 * 4
    cache = kv4.empty(3, 2, 16, 64, device="cpu")
    assert tuple(cache.shape) == (3, 2, 2, 16, 40) and cache.dtype == torch.uint8
    with pytest.raises(RuntimeError):
        kv4.empty(3, 2, 24, 64, device="cpu")
    with pytest.raises(ValueError):        # no CPU form
        kv4.read(cache, torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32),
                 torch.tensor([0, 1], dtype=torch.int32), k_out=torch.zeros(2, 1, 64))


def test_plain_form_of_the_format():
    """The oracle itself: levels within half a step, extremes, constants, and the layout's places."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((500, 128)).astype(np.float32) * 10 ** rng.uniform(-3, 3, (500, 1)).astype(np.float32)
    levels, pairs = KP.quantise(x)
    back = KP.value_of(levels, pairs)
    scale = (pairs[..., 0].astype(np.uint32) << 16).view(np.float32).repeat(KP.GROUP, -1)
    assert np.all(np.abs(back - x) <= scale * (0.5 + 2.0 ** -15)) and levels.max() == 15
    assert np.all(KP.value_of(*KP.quantise(np.full((1, 64), -3.25, np.float32))) == -3.25)
    for d in (64, 128):
        for values in (False, True):
            for off in range(8):
                assert len({KP.place(c, off, d, values) for c in range(d)}) == d


# -------------------------------------------------------------------------------------- GPU: helpers

def _special(x, rng):
    """Rows where a group is constant, zero, tiny, huge, holds -0, NaN or infinities."""
    flat = x.reshape(-1, 32)
    n = flat.shape[0]
    for i, fill in enumerate((0.0, -0.0, 1.5, -7.0, 1e-38, 3e38)):
        flat[(3 + 7 * i) % n] = fill
    flat[5 % n, 3] = np.nan
    flat[11 % n, 31] = np.inf
    flat[12 % n, 0] = -np.inf
    flat[16 % n, 1], flat[16 % n, 2] = 3.3e38, -3.3e38          # the range overflows
    flat[19 % n] *= 1e-39                                         # denormals: stored as a constant
    flat[20 % n] = np.where(rng.random(32) < 0.5, -0.0, 0.0)
    return x


class Batch:
    """Sequences of given lengths and new tokens on a pool of shuffled pages, on the host and the GPU."""

    def __init__(self, lens, new, page, hkv, d, seed=0, spare=0, first=0, extra=2, fill=0xFF):
        rng = np.random.default_rng(seed)
        self.lens, self.new, self.page, self.hkv, self.d = lens, new, page, hkv, d
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + extra
        order = rng.permutation(self.pages)
        self.table = np.full((len(lens), max(need + [1]) + 1), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cu = (first + np.concatenate([[0], np.cumsum(new)])).astype(np.int32)
        self.total = int(self.cu[-1]) + spare
        # what no token has written reads as NaN (0xFFFF pairs)
        self.cache = np.full((self.pages, hkv, 2, page, 5 * d // 8), fill, np.uint8)

    def gpu(self):
        self.g_cache = torch.from_numpy(self.cache).cuda()
        self.g = [torch.from_numpy(np.asarray(x, np.int32)).cuda() for x in (self.table, self.lens, self.cu)]
        return self

    def put(self, b, pos, k, v):
        """One token of sequence b into the host's cache (k, v [Hkv, d]); what it stands for."""
        page, off = self.table[b, pos // self.page], pos % self.page
        return [[KP.put_token(self.cache, page, h, side, off, x[h]) for h in range(self.hkv)]
                for side, x in ((0, k), (1, v))]

    def fill(self, rng, shift=1.0):
        """Every token of every sequence."""
        bias = rng.standard_normal((self.hkv, self.d)) * shift
        for b, n in enumerate(self.lens):
            for pos in range(n):
                x = rng.standard_normal((2, self.hkv, self.d))
                self.put(b, pos, (x[0] + bias).astype(np.float32), x[1].astype(np.float32))
        return self


def _fast_fill(batch, rng, shift=1.0):
    """As Batch.fill, but with random levels and pairs (for longer contexts)."""
    d, page, n = batch.d, batch.page, batch.pages
    flat = batch.cache.reshape(n, batch.hkv, 2, -1)
    flat[..., :page * d // 2] = rng.integers(0, 256, (n, batch.hkv, 2, page * d // 2), np.uint8)
    scale = rng.uniform(0.1, 0.3, (n, batch.hkv, 2, page, d // 32)).astype(np.float32)
    low = (-7.5 * scale + rng.normal(0, 0.3 * shift, scale.shape)).astype(np.float32)
    pairs = np.stack([scale, low], -1).view(np.uint32) >> 16
    flat[..., page * d // 2:] = pairs.astype(np.uint16).view(np.uint8).reshape(n, batch.hkv, 2, -1)
    return batch


def _rows(rng, heads, total, d, dtype, token_major, scale=1.0, pad=0):
    x = torch.from_numpy(rng.standard_normal((total, heads, d + pad)).astype(np.float32) * np.float32(scale))
    x = x.to(DT[dtype]).cuda()[..., :d].transpose(0, 1)
    return x if token_major else x.contiguous()


def _status(kv4):
    from block_sparse_attention_sbsa_b200 import sbsa
    return sbsa.get_status()


def _tolerance(o, size, span, dtype, n, d):
    if dtype == "bf16":
        return 2.0 ** -8 * np.abs(o) + 2.0 ** -11 * span * (2 + 2 * size) + 1e-30
    return span * (2 * (d + 18) * 2.0 ** -23 * size + 2.0 ** -21 + 2.0 ** -23 * (64 + n / 64)) + 1e-30


def _check(kv4, batch, q, out, before, scale=None, idx=None, cnt=None, block=0, dtype="bf16"):
    """The rows of sequences against float64, the others as they were."""
    want, size, span = KP.attend(KP.decode(batch.cache), q.float().cpu().numpy(), batch.table, batch.lens,
                                 batch.cu, scale, idx, cnt, block)
    got = out.float().cpu().numpy()
    mine = np.zeros(batch.total, bool)
    mine[batch.cu[0]:batch.cu[-1]] = True
    assert np.array_equal(got[:, ~mine], before.float().cpu().numpy()[:, ~mine])
    err = np.abs(got - want)[:, mine]
    tol = _tolerance(want, size, span, dtype, max(batch.lens), batch.d)[:, mine]
    assert np.isfinite(got[:, mine]).all()
    assert (err <= tol).all(), (err.max(), (err / tol).max(), np.argwhere(err > tol)[:5])


# --------------------------------------------------------------------------------- GPU: append, read

@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,token_major", [("bf16", True), ("fp32", False)])
def test_append_and_read_are_the_format(kv4, cuda, page, d, dtype, token_major):
    rng = np.random.default_rng(page + d)
    lens, new = [page * 2 + 3, 5, 1, 70, 0, page], [page + 9, 0, 1, 70, 0, page]
    b = Batch(lens, new, page, 3, d, seed=d, spare=4, first=2, fill=0xA5).gpu()
    x = _special(rng.standard_normal((2, 3, b.total, d)).astype(np.float32) * 2, rng)
    x = torch.from_numpy(x).to(DT[dtype])
    k, v = (t.transpose(0, 1).contiguous().cuda().transpose(0, 1) if token_major else t.cuda() for t in x)
    ks, vs = (torch.full((3, b.total, d), 9.0, dtype=DT[dtype], device="cuda") for _ in range(2))
    kv4.append(b.g_cache, k, v, *b.g, k_stored=ks, v_stored=vs)
    xs = x.float().numpy()
    stored = np.full((2, 3, b.total, d), 9.0, np.float32)
    for s, n in enumerate(lens):
        for t in range(b.cu[s], b.cu[s + 1]):
            stored[:, :, t] = b.put(s, n - b.cu[s + 1] + t, xs[0][:, t], xs[1][:, t])
    assert np.array_equal(b.g_cache.cpu().numpy(), b.cache)          # the rest of the cache as it was
    stored = torch.from_numpy(stored).to(DT[dtype])
    for got, want in ((ks, stored[0]), (vs, stored[1])):
        assert torch.equal(got.cpu().nan_to_num(nan=77.0), want.nan_to_num(nan=77.0))
    ko, vo = (torch.full((3, b.total, d), 9.0, dtype=DT[dtype], device="cuda") for _ in range(2))
    kv4.read(b.g_cache, *b.g, k_out=ko, v_out=vo)
    for got, want in ((ko, ks), (vo, vs)):
        assert torch.equal(got.nan_to_num(nan=77.0), want.nan_to_num(nan=77.0))
    only = torch.empty(3, b.total, d, dtype=torch.float32, device="cuda")
    kv4.read(b.g_cache, *b.g, v_out=only)
    mine = slice(int(b.cu[0]), int(b.cu[-1]))
    assert torch.equal(only[:, mine].to(DT[dtype]).nan_to_num(nan=77.0), vs[:, mine].nan_to_num(nan=77.0))
    assert _status(kv4) == 0


@pytest.mark.gpu
def test_places_out_of_range_are_skipped_and_reported(kv4, cuda):
    page, d = 32, 64
    b = Batch([40, 20, 10], [4, 3, 12], page, 2, d, seed=1).gpu()      # 12 new of 10 tokens: two before the first
    b.g[0][0, 1] = b.pages                                              # sequence 0's second page
    b.g[0][1, 0] = -5
    rng = np.random.default_rng(2)
    k, v = (_rows(rng, 2, b.total, d, "fp32", False) for _ in range(2))
    before = b.g_cache.clone()
    kv4.append(b.g_cache, k, v, *b.g)
    assert _status(kv4) == 6
    for t in range(9, 19):
        b.put(2, t - 9, k[:, t].cpu().numpy(), v[:, t].cpu().numpy())
    assert np.array_equal(b.g_cache.cpu().numpy(), b.cache) and not torch.equal(before, b.g_cache)
    out = torch.full((2, b.total, d), 9.0, device="cuda")
    kv4.read(b.g_cache, *b.g, k_out=out)
    assert _status(kv4) == 6
    assert (out[:, :9] == 0).all() and out[:, 9:].abs().max() > 0
    b.g[1].fill_(10 ** 9)                                               # lengths beyond the table
    kv4.read(b.g_cache, *b.g, k_out=out)
    assert _status(kv4) == 6
    b.g[1].fill_(-3)
    kv4.read(b.g_cache, *b.g, k_out=out)
    assert _status(kv4) == 6 and (out == 0).all()


# -------------------------------------------------------------------------------------- GPU: attend

@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (5, 1), (16, 2), (24, 2), (36, 2)])
@pytest.mark.parametrize("d,page,dtype", [(64, 16, "fp32"), (64, 128, "bf16"), (128, 32, "fp32"),
                                          (128, 64, "bf16")])
def test_attend_steps(kv4, cuda, hq, hkv, d, page, dtype):
    """One token a sequence: lengths around tiles and pages, an empty sequence, one without a row."""
    rng = np.random.default_rng(hq * 1000 + d)
    lens = [1, 15, 16, 17, 127, 128, 129, 300, 0, 513]
    b = _fast_fill(Batch(lens, [1] * 8 + [0, 1], page, hkv, d, seed=hq, spare=3, first=1), rng).gpu()
    q = _rows(rng, hq, b.total, d, dtype, True, 1.5)
    out = torch.full_like(q, 3.0)
    before = out.clone()
    assert kv4.attend(b.g_cache, q, *b.g, 1, out=out) is out
    assert _status(kv4) == 0
    _check(kv4, b, q, out, before, dtype=dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d,page,dtype", [(4, 4, 64, 16, "bf16"), (8, 1, 128, 64, "bf16"),
                                                 (6, 2, 128, 32, "fp32"), (10, 2, 64, 64, "bf16"),
                                                 (32, 2, 128, 128, "bf16")])
@pytest.mark.parametrize("new", [(1, 2, 3, 4), (7, 0, 5, 2), (40, 17, 33, 9), (129, 1, 64, 200)])
def test_attend_chunks(kv4, cuda, hq, hkv, d, page, dtype, new):
    """Several rows a sequence: the causal edge inside tiles, whole sequences new, rows of other sequences."""
    rng = np.random.default_rng(sum(new) + hq)
    lens = [new[0], 130 + new[1], 2 * page + new[2], 400 + new[3]]
    b = _fast_fill(Batch(lens, list(new), page, hkv, d, seed=hq, spare=2), rng).gpu()
    q = _rows(rng, hq, b.total, d, dtype, True, 1.2, pad=64 if d == 64 else 0)
    out = torch.zeros(hq, b.total, d, dtype=DT[dtype], device="cuda")
    kv4.attend(b.g_cache, q, *b.g, max(new), out=out, sm_scale=0.11)
    assert _status(kv4) == 0
    _check(kv4, b, q, out, torch.zeros_like(out), scale=float(np.float32(0.11)), dtype=dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("d,most", [(64, 1), (128, 5), (64, 150), (128, 90)])
def test_attend_many_items_a_cta(kv4, cuda, d, most):
    """Enough sequences of mixed sizes that every CTA walks several items, whole and shared, with one
    and two query tiles, of one and many token tiles, in mixed order."""
    rng = np.random.default_rng(most)
    seqs = 160 if most < 9 else 36
    lens = [int(x) for x in np.exp(rng.uniform(np.log(3), np.log(1500 if most < 9 else 2500), seqs))]
    new = [min(n, int(rng.integers(0, most + 1)) if rng.random() < 0.5 else most) for n in lens]
    b = _fast_fill(Batch(lens, new, 64, 2, d, seed=most), rng).gpu()
    q = _rows(rng, 8, b.total, d, "bf16", True, 1.5)
    out = torch.zeros_like(q)
    kv4.attend(b.g_cache, q, *b.g, max(new), out=out)
    assert _status(kv4) == 0
    _check(kv4, b, q, out, torch.zeros_like(out))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("most", [8, 9, 12, 13, 32, 33])
def test_attend_at_the_limits_between_kernels(kv4, cuda, d, most):
    """32, 36, 48 and 52 rows of a kv head (the kernels change after 32 or 48), 128 and 132 (one query tile
    and two), with contexts that end at, before and behind a tile of 128 tokens."""
    rng = np.random.default_rng(most + d)
    lens = [128 + most, 127, 129, 640, 33, 1411]
    new = [most, most, 1, most - 1, min(most, 33), most]
    b = _fast_fill(Batch(lens, new, 32, 2, d, seed=most), rng).gpu()
    q = _rows(rng, 8, b.total, d, "bf16", True, 1.5)
    out = torch.zeros_like(q)
    kv4.attend(b.g_cache, q, *b.g, most, out=out)
    assert _status(kv4) == 0
    _check(kv4, b, q, out, torch.zeros_like(out))


@pytest.mark.gpu
@pytest.mark.parametrize("list_heads", ["kv", "q"])
@pytest.mark.parametrize("block,page,d,dtype", [(64, 64, 128, "bf16"), (128, 16, 64, "fp32"), (128, 128, 128, "bf16"),
                                                (64, 32, 64, "bf16")])
def test_attend_listed_blocks(kv4, cuda, list_heads, block, page, d, dtype):
    rng = np.random.default_rng(block + page)
    hq, hkv = 6, 2
    lens, new = [700, 64, 1000, 129, 90], [1, 1, 3, 2, 1]
    b = _fast_fill(Batch(lens, new, page, hkv, d, seed=3), rng).gpu()
    heads, width = (hkv if list_heads == "kv" else hq), 5
    idx = np.full((5, heads, width), -1, np.int32)
    cnt = np.zeros((5, heads), np.int32)
    for s, n in enumerate(lens):
        nb = -(-n // block)
        for h in range(heads):
            c = min(nb, int(rng.integers(1, width + 1)))
            idx[s, h, :c] = np.sort(rng.choice(nb, c, replace=False))
            cnt[s, h] = c
    idx[0, 0, :3], cnt[0, 0] = (2, 2, 4), 3         # a block twice
    cnt[2, 1] = 0                                     # a list without a block: rows of zeros
    q = _rows(rng, hq, b.total, d, dtype, False, 1.5)
    out = torch.full_like(q, 3.0)
    before = out.clone()
    kv4.attend(b.g_cache, q, *b.g, 3, idx=torch.from_numpy(idx).cuda(), cnt=torch.from_numpy(cnt).cuda(),
               block_size=block, out=out)
    assert _status(kv4) == 0
    _check(kv4, b, q, out, before, idx=idx, cnt=cnt, block=block, dtype=dtype)


@pytest.mark.gpu
def test_attend_reports_what_is_out_of_range(kv4, cuda):
    rng = np.random.default_rng(5)
    page, d, hkv, hq = 16, 64, 1, 2
    b = _fast_fill(Batch([100, 50, 30], [1, 1, 4], page, hkv, d, seed=5), rng).gpu()
    q = _rows(rng, hq, b.total, d, "bf16", False)
    idx = np.array([[[0, 9, 1, -2]], [[0, 0, 0, 0]], [[0, 0, 0, 0]]], np.int32)      # blocks 9, -2: outside
    cnt = np.array([[4], [1], [1]], np.int32)
    out = torch.zeros_like(q)
    kv4.attend(b.g_cache, q, *b.g, 4, idx=torch.from_numpy(idx).cuda(), cnt=torch.from_numpy(cnt).cuda(),
               block_size=64, out=out)
    assert _status(kv4) == 6
    _check(kv4, b, q, out, torch.zeros_like(q), idx=idx, cnt=cnt, block=64)
    # a page number outside the cache: its tokens are not seen
    b.g[0][0, 2] = b.pages + 7
    kv4.attend(b.g_cache, q, *b.g, 4, out=out)
    assert _status(kv4) == 6
    dec = KP.decode(b.cache)
    k, v = (x[:, 0].astype(np.float64) for x in KP.tokens(dec, b.table[0], 100))
    keep = np.r_[0:32, 48:100]
    for h in range(hq):
        s = k[keep] @ q[h, 0].double().cpu().numpy() / 8
        p = np.exp(s - s.max())
        want = p @ v[keep] / p.sum()
        assert np.abs(out[h, 0].double().cpu().numpy() - want).max() < 0.05
    # more rows than max_new: those beyond are 0 and reported
    b.g[0].copy_(torch.from_numpy(b.table))
    out.fill_(5.0)
    kv4.attend(b.g_cache, q, *b.g, 2, out=out)
    assert _status(kv4) == 6
    assert (out[:, 4:6] == 0).all() and (out[:, :4] != 0).any(dim=-1).all()
    # rows before a sequence's first token
    b.g[1][2] = 2
    out.fill_(5.0)
    kv4.attend(b.g_cache, q, *b.g, 4, out=out)
    assert _status(kv4) == 6 and (out[:, 2:4] == 0).all() and torch.isfinite(out).all()


@pytest.mark.gpu
def test_attend_many_rows_reports_what_is_out_of_range(kv4, cuda):
    """The same for a chunk of more rows than the few-row kernel takes: a page outside the cache in the middle
    of a tile, rows beyond max_new, rows before the sequence's first token, in two query tiles."""
    rng = np.random.default_rng(6)
    page, d, hkv, hq, n, new = 16, 64, 1, 4, 300, 60
    b = _fast_fill(Batch([n, 90], [new, new], page, hkv, d, seed=6), rng).gpu()
    q = _rows(rng, hq, b.total, d, "bf16", True)
    out = torch.zeros_like(q)
    b.g[0][0, 9] = b.pages + 3
    kv4.attend(b.g_cache, q, *b.g, new, out=out)
    assert _status(kv4) == 6
    k, v = (x[:, 0].astype(np.float64) for x in KP.tokens(KP.decode(b.cache), b.table[0], n))
    for h in range(hq):
        for t in (0, 31, 59):
            keep = np.array([u for u in range(n - new + t + 1) if not 144 <= u < 160])
            s = k[keep] @ q[h, t].double().cpu().numpy() / 8
            p = np.exp(s - s.max())
            assert np.abs(out[h, t].double().cpu().numpy() - p @ v[keep] / p.sum()).max() < 0.02
    b.g[0].copy_(torch.from_numpy(b.table))
    out.fill_(5.0)
    kv4.attend(b.g_cache, q, *b.g, 50, out=out)
    assert _status(kv4) == 6
    assert (out[:, 50:60] == 0).all() and (out[:, 110:] == 0).all()
    _check_rows = np.r_[0:50, 60:110]
    want, size, span = KP.attend(KP.decode(b.cache), q.float().cpu().numpy(), b.table, b.lens, b.cu)
    err = np.abs(out.float().cpu().numpy() - want)[:, _check_rows]
    assert (err <= _tolerance(want, size, span, "bf16", n, d)[:, _check_rows]).all()
    b.g[1][1] = 20
    out.fill_(5.0)
    kv4.attend(b.g_cache, q, *b.g, new, out=out)
    assert _status(kv4) == 6 and (out[:, 60:100] == 0).all() and (out[:, 100:] != 0).any(dim=-1).all()
    b.g[1].fill_(0)
    kv4.attend(b.g_cache, q, *b.g, new, out=out)
    assert _status(kv4) == 6 and (out == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_attend_long_contexts_have_no_drift(kv4, cuda, dtype):
    """Over many tokens the output is a small mean of large values, so an error that does not average out
    shows.  Each row's error, over channels, has a 2-norm below: fp32, 2^-22 of the values' (a bit of the
    weights' two parts) plus 2^-21 of the output's; bf16, its rounding 2^-9 of the output in the mean
    (uniform up to 2^-8) plus 2^-11 of the values' over the square root of the tokens that count, plus
    2^-18 of the values' for sums in 18 bits."""
    d, n, hq = 128, 60000, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v, q = (torch.randn(h, t, d, generator=g, device="cuda").to(DT[dtype]) for h, t in ((1, n), (1, n), (hq, 1)))
    pages = -(-n // 64)
    cache = kv4.empty(pages, 1, 64, d)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None]
    lens, cu, one = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([n], [0, n], [0, 1]))
    kv4.append(cache, k, v, table, lens, cu)
    kr, vr = (torch.empty(1, n, d, device="cuda") for _ in range(2))
    kv4.read(cache, table, lens, cu, k_out=kr, v_out=vr)
    o = kv4.attend(cache, q, table, lens, one, 1)[:, 0].double()
    p = torch.softmax(q[:, 0].double() @ kr[0].double().T / d ** 0.5, -1)
    want = p @ vr[0].double()
    err, size = (o - want).norm(dim=-1), vr[0].double().norm(dim=-1).mean()
    if dtype == "fp32":
        assert (err <= 2.0 ** -22 * size + 2.0 ** -21 * want.norm(dim=-1)).all(), err / size
    else:
        spread = p.square().sum(-1).sqrt()
        assert (err <= 2.0 ** -9 * want.norm(dim=-1) + (2.0 ** -11 * spread + 2.0 ** -18) * size).all(), err / size


@pytest.mark.gpu
def test_two_streams_at_once(kv4, cuda):
    """Calls that overlap, few and many rows, each with its own workspace."""
    rng = np.random.default_rng(13)
    b = _fast_fill(Batch([3000, 500, 1200], [1, 1, 1], 64, 2, 128, seed=13), rng).gpu()
    c = _fast_fill(Batch([2000, 700], [300, 41], 32, 2, 128, seed=14), rng).gpu()
    q, r = _rows(rng, 8, 3, 128, "bf16", True), _rows(rng, 8, c.total, 128, "bf16", True)
    one, two = kv4.attend(b.g_cache, q, *b.g, 1), kv4.attend(c.g_cache, r, *c.g, 300)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for i, s in enumerate(streams):
            got.append(kv4.attend(b.g_cache, q, *b.g, 1, stream=s) if i % 2 else
                       kv4.attend(c.g_cache, r, *c.g, 300, stream=s))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, one if i % 2 else two)
    assert _status(kv4) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 70])
def test_attend_spread_of_magnitudes(kv4, cuda, new):
    """Values and keys whose size differs by 2^16 between tokens and groups, a token with a NaN
    group, constant groups, and logits far from zero."""
    rng = np.random.default_rng(11)
    d, hkv, hq, n = 128, 1, 4, 300
    b = Batch([n], [new], 64, hkv, d, seed=4)
    for pos in range(n):
        x = rng.standard_normal((2, 1, d)).astype(np.float32)
        x[1] *= np.float32(2.0) ** rng.integers(-10, 7, (1, d // 32)).repeat(32, 1)
        x[0] *= np.float32(2.0) ** rng.integers(-3, 2, (1, d // 32)).repeat(32, 1)
        if pos % 7 == 0:
            x[1, :, 32:64] = 3.0
        b.put(0, pos, x[0], x[1])
    b.gpu()
    q = _rows(rng, hq, new, d, "bf16", False, 6.0)
    out = torch.zeros_like(q)
    kv4.attend(b.g_cache, q, *b.g, new, out=out)
    _check(kv4, b, q, out, torch.zeros_like(q))
    x = rng.standard_normal((2, 1, d)).astype(np.float32)
    x[1, 0, 40] = np.nan
    b.put(0, 5, x[0], x[1])
    b.gpu()
    kv4.attend(b.g_cache, q, *b.g, new, out=out)
    assert torch.isnan(out[..., 32:64]).all() and torch.isfinite(out[..., :32]).all() \
        and torch.isfinite(out[..., 64:]).all()
    want, size, span = KP.attend(KP.decode(b.cache), q.float().cpu().numpy(), b.table, b.lens, b.cu)
    fin = np.r_[0:32, 64:128]
    tol = _tolerance(want, size, np.nan_to_num(span, nan=512.0), "bf16", n, d)
    assert (np.abs(out.float().cpu().numpy() - want)[..., fin] <= np.maximum(tol, 0.02)[..., fin] + 2.0 ** -7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,dtype", [(3, "bf16"), (3, "fp32"), (70, "bf16")])
def test_attend_a_nan_key_is_met_only_by_rows_that_see_it(kv4, cuda, d, new, dtype):
    """A key with a NaN in one group, among the new tokens: the rows before it stay what they are, the
    others are NaN; so do the value's channels of its group alone with a NaN value."""
    rng = np.random.default_rng(new + d)
    n, at = 300, 300 - new + new // 2
    b = _fast_fill(Batch([n], [new], 64, 1, d, seed=8), rng)
    q = _rows(rng, 4, new, d, dtype, True, 1.2)
    want, size, span = KP.attend(KP.decode(b.cache), q.float().cpu().numpy(), b.table, b.lens, b.cu)
    tol = _tolerance(want, size, span, dtype, n, d)
    first = at - (n - new)  # the first row that sees it
    for side in (0, 1):
        kept = b.cache.copy()
        x = rng.standard_normal((2, 1, d)).astype(np.float32)
        x[side, 0, 33] = np.nan
        b.put(0, at, x[0], x[1])
        b.gpu()
        out = torch.zeros(4, new, d, dtype=DT[dtype], device="cuda")
        kv4.attend(b.g_cache, q, *b.g, new, out=out)
        got = out.float().cpu().numpy()
        assert (np.abs(got - want)[:, :first] <= tol[:, :first]).all()
        assert np.isnan(got[:, first:, slice(None) if side == 0 else slice(32, 64)]).all()
        if side:
            assert np.isfinite(np.delete(got[:, first:], np.r_[32:64], axis=2)).all()
        b.cache[...] = kept


@pytest.mark.gpu
def test_other_stream_graph_and_new_lengths(kv4, cuda):
    """On a stream of its own; captured, and replayed with other lengths, tables and queries; two graphs
    on one workspace."""
    rng = np.random.default_rng(8)
    hq, hkv, d, page = 8, 2, 128, 32
    b = _fast_fill(Batch([900, 333], [1, 1], page, hkv, d, seed=8), rng).gpu()
    k, v = (_rows(rng, hkv, 2, d, "bf16", True) for _ in range(2))
    q = _rows(rng, hq, 2, d, "bf16", True, 1.5)
    ws = torch.empty(kv4.attend_workspace_bytes(_params(kv4)), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [torch.zeros_like(q) for _ in range(3)]
    kv4.attend(b.g_cache, q, *b.g, 1, out=outs[0], stream=side)
    side.synchronize()
    _check(kv4, b, q, outs[0], torch.zeros_like(q))
    graphs = []
    for o in outs[1:]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kv4.append(b.g_cache, k, v, *b.g)
            kv4.attend(b.g_cache, q, *b.g, 1, out=o, workspace=ws)
        graphs.append(g)
    for step in range(3):
        b.lens = [900 + step, 333 - 100 * step]
        for s, n in enumerate(b.lens):
            if b.table[s, (n - 1) // page] < 0:
                b.table[s, (n - 1) // page] = b.table[s].max() if False else (set(range(b.pages)) - set(b.table.ravel())).pop()
        b.g[1].copy_(torch.tensor(b.lens, dtype=torch.int32))
        b.g[0].copy_(torch.from_numpy(b.table))
        q.copy_(_rows(rng, hq, 2, d, "bf16", True, 1.5))
        k.copy_(_rows(rng, hkv, 2, d, "bf16", True))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for s, n in enumerate(b.lens):
            b.put(s, n - 1, k[:, s].float().cpu().numpy(), v[:, s].float().cpu().numpy())
        for o in outs[1:]:
            _check(kv4, b, q, o, torch.zeros_like(q))
    assert _status(kv4) == 0


@pytest.mark.gpu
def test_results_do_not_change_between_runs(kv4, cuda):
    rng = np.random.default_rng(9)
    b = _fast_fill(Batch([5000, 77, 2049], [3, 1, 2], 64, 2, 128, seed=9), rng).gpu()
    q = _rows(rng, 8, b.total, 128, "bf16", True)
    one = kv4.attend(b.g_cache, q, *b.g, 3)
    for _ in range(5):
        assert torch.equal(one, kv4.attend(b.g_cache, q, *b.g, 3))


@pytest.mark.gpu
def test_pages_behind_four_gigabytes(kv4, cuda):
    """A cache of more than 2^32 bytes: tokens in its last pages."""
    d, page, hkv = 128, 128, 8
    pages = (1 << 32) // (hkv * 2 * page * 80) + 40
    cache = torch.empty(pages, hkv, 2, page, 80, dtype=torch.uint8, device="cuda")
    assert cache.numel() > 1 << 32
    rng = np.random.default_rng(10)
    n = 300
    small = Batch([n], [n], page, hkv, d, seed=1, extra=0)
    small.gpu()
    table = torch.tensor([[pages - 1, pages - 7, pages - 3]], dtype=torch.int32, device="cuda")
    k, v = (_rows(rng, hkv, n, d, "bf16", True) for _ in range(2))
    kv4.append(cache, k, v, table, *small.g[1:])
    kv4.append(small.g_cache, k, v, *small.g)
    small.cache = small.g_cache.cpu().numpy()
    ko = torch.empty(hkv, n, d, dtype=torch.float32, device="cuda")
    want = torch.empty_like(ko)
    kv4.read(cache, table, *small.g[1:], k_out=ko)
    kv4.read(small.g_cache, *small.g, k_out=want)
    assert torch.equal(ko, want)
    for rows in (1, n):
        cu = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        q = _rows(rng, 16, rows, d, "bf16", True)
        one = kv4.attend(cache, q, table, small.g[1], cu, rows)
        two = kv4.attend(small.g_cache, q, small.g[0], small.g[1], cu, rows)
        assert torch.equal(one, two)
    assert _status(kv4) == 0


@pytest.mark.gpu
def test_prefill_then_generate(kv4, cuda):
    """The operators as they are used: a prefill over what the cache stands for, tokens appended and attended
    one at a time, densely and over the prompt's last block list, and the cache read back for pooling."""
    from block_sparse_attention_sbsa_b200 import sbsa
    rng = np.random.default_rng(12)
    hq, hkv, d, n, block = 8, 2, 128, 1000, 128
    p = sbsa.make_params(n_q_heads=hq, n_kv_heads=hkv, seq_len=n, head_dim=d, block_size=block,
                         dtype="bf16", select_mode="topk", top_k=3, group_shared=True)
    b = Batch([n + 40], [n + 40], 64, hkv, d, seed=12).gpu()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    q, k, v = (_rows(rng, h, n, d, "bf16", True) for h in (hq, hkv, hkv))
    ks, vs = (torch.empty(hkv, n, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kv4.append(b.g_cache, k, v, b.g[0], lens, cu, k_stored=ks, v_stored=vs)
    o, idx, cnt, _ = sbsa.prefill(p, q.contiguous(), ks, vs)
    # the last rows of the prefill are those that attention over the cache gives for the same list
    tail = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    got = kv4.attend(b.g_cache, q[:, -20:], b.g[0], lens, tail, 20, idx=idx[:, -1:].transpose(0, 1).contiguous(),
                     cnt=cnt[:, -1:].transpose(0, 1).contiguous(), block_size=block)
    assert (got.float() - o[:, -20:].float()).abs().max() < 2e-2
    # read back, pooled again: the same centroids
    ko = torch.empty_like(ks)
    kv4.read(b.g_cache, b.g[0], lens, cu, k_out=ko)
    assert torch.equal(ko, ks)
    assert torch.equal(sbsa.pool_blocks(p, ko)[0], sbsa.pool_blocks(p, ks)[0])
    # generation
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for step in range(4):
        lens += 1
        q1, k1, v1 = (_rows(rng, h, 1, d, "bf16", True) for h in (hq, hkv, hkv))
        kv4.append(b.g_cache, k1, v1, b.g[0], lens, one)
        o1 = kv4.attend(b.g_cache, q1, b.g[0], lens, one, 1)
        b.cache, b.lens, b.cu, b.total = b.g_cache.cpu().numpy(), [n + 1 + step], np.array([0, 1]), 1
        _check(kv4, b, q1, o1, torch.zeros_like(o1))
    assert _status(kv4) == 0


@pytest.mark.gpu
def test_binding_refuses(kv4, cuda):
    b = Batch([10, 20], [1, 2], 16, 2, 64).gpu()
    rng = np.random.default_rng(0)
    k, q = _rows(rng, 2, 3, 64, "bf16", True), _rows(rng, 4, 3, 64, "bf16", True)
    t, lens, cu = b.g
    bad = [
        lambda: kv4.append(b.g_cache, k, k, t, lens, cu[:2]),
        lambda: kv4.append(b.g_cache, k, k, t.long(), lens, cu),
        lambda: kv4.append(b.g_cache, k, k, t, lens.cpu(), cu),
        lambda: kv4.append(b.g_cache, k, k.float(), t, lens, cu),
        lambda: kv4.append(b.g_cache, k.half(), k.half(), t, lens, cu),
        lambda: kv4.append(b.g_cache, k, k[:, :2], t, lens, cu),
        lambda: kv4.append(b.g_cache, k[..., ::2], k[..., ::2], t, lens, cu),
        lambda: kv4.append(b.g_cache, k, k, t, lens, cu, k_stored=k),
        lambda: kv4.append(b.g_cache[:, :, :1], k, k, t, lens, cu),
        lambda: kv4.read(b.g_cache, t, lens, cu),
        lambda: kv4.read(b.g_cache, t, lens, cu, k_out=k),
        lambda: kv4.attend(b.g_cache, q[:3], t, lens, cu, 2),
        lambda: kv4.attend(b.g_cache, q, t, lens, cu, 0),
        lambda: kv4.attend(b.g_cache, q, t, lens, cu, 2, out=q[:, :2]),
        lambda: kv4.attend(b.g_cache, q, t, lens, cu, 2, idx=torch.zeros(2, 2, 1, dtype=torch.int32, device="cuda")),
        # (a table of 160 tokens, which needs a workspace)
        lambda: kv4.attend(b.g_cache, q, t.repeat(1, 5)[:, :10].contiguous(), lens, cu, 2,
                           workspace=torch.empty(8, dtype=torch.uint8, device="cuda")),
        lambda: kv4.attend(b.g_cache, q, t, lens, cu, 2, workspace=torch.empty(8, device="cuda")),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, RuntimeError)):
            call()
            pytest.fail(f"call {i} was taken")
