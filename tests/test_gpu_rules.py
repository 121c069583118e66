"""Token history and logit rules on the GPU against their plain 64-bit forms."""
import numpy as np
import pytest
import torch

import _plain_rules as plain
import speculative_decoding_verification_93_b200 as sv

pytestmark = pytest.mark.gpu

DT = {"float32": torch.float32, "bfloat16": torch.bfloat16}


def dev(x, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(x)).to("cuda", dtype)


def new_status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# History.
# ---------------------------------------------------------------------------
def check_history(h, want):
    torch.cuda.synchronize()
    assert np.array_equal(h.output_counts.cpu().numpy(), want.counts)
    assert np.array_equal(h.output_bits.cpu().numpy(), plain.pack(want.counts > 0))
    assert np.array_equal(h.prompt_bits.cpu().numpy(), plain.pack(want.prompt))


@pytest.mark.parametrize("B,S,V", [(1, 1, 1), (1, 1, 32), (3, 7, 33), (4, 5, 1000), (2, 5000, 64),
                                   (70, 9, 129280), (1, 20000, 129280)])
def test_history_add(B, S, V):
    rng = np.random.default_rng(B + S + V)
    h, want = sv.TokenHistory.empty(B + 2, V, "cuda"), plain.History(B + 2, V)
    for step in range(3):
        tokens = rng.integers(0, V, (B, S)).astype(np.int32)
        tokens[:, S // 2:] = tokens[:, :1]                   # the same token many times over
        lens = rng.integers(0, S + 1, B).astype(np.int32)
        st = new_status()
        prompt = step == 0
        sv.sv_history_add(h, dev(tokens), dev(lens),
                          sv.SV_HISTORY_PROMPT if prompt else sv.SV_HISTORY_OUTPUT, status=st)
        for b in range(B):
            want.add(b, tokens[b, :lens[b]], prompt)
        check_history(h, want)
        assert int(st) == 0


def test_history_takes_verification_results_and_marks_bad_data():
    V, K = 50, 4
    h, want = sv.TokenHistory.empty(3, V, "cuda"), plain.History(3, V)
    tokens = np.array([[3, 3, 49, -1, -1], [-1] * 5, [0, 1, 2, 3, 4], [7, 8, 9, 10, 11],
                       [5, 5, 5, 5, 5], [5, 50, 6, -3, 6]], np.int32)
    acc = np.array([2, -1, 4, 5, 1, 4], np.int32)      # row 3: six tokens of five, refused
    slots = np.array([2, 0, 0, 1, 3, 2], np.int32)     # rows 0 and 5 share a slot, row 4 has none
    st = new_status()
    sv.sv_history_add(h, dev(tokens), dev(acc), slots=dev(slots), extra=1, status=st)
    want.add(2, [3, 3, 49, 5, 6, 6])
    want.add(0, [0, 1, 2, 3, 4])
    check_history(h, want)
    assert int(st) == sv.SV_ROW_BAD_LENGTH | sv.SV_ROW_BAD_SLOT | sv.SV_ROW_BAD_TOKEN
    # without lens: every entry
    sv.sv_history_add(h, dev(tokens[2:3]), kind=sv.SV_HISTORY_PROMPT)
    want.add(0, tokens[2], prompt=True)
    check_history(h, want)


@pytest.mark.parametrize("V", [1, 32, 1000, 50001])
def test_history_reset(V):
    rng = np.random.default_rng(V)
    R = 6
    h, want = sv.TokenHistory.empty(R, V, "cuda"), plain.History(R, V)
    tokens = rng.integers(0, V, (R, 300)).astype(np.int32)
    tokens[:, 0] = V - 1
    for kind in (sv.SV_HISTORY_PROMPT, sv.SV_HISTORY_OUTPUT):
        sv.sv_history_add(h, dev(tokens), kind=kind)
    for b in range(R):
        want.add(b, tokens[b])
        want.add(b, tokens[b], prompt=True)
    st = new_status()
    sv.sv_history_reset(h, dev(np.array([4, 1, 4, -1, R], np.int32)), status=st)
    for b in (1, 4):
        want.counts[b] = 0
        want.prompt[b] = False
    check_history(h, want)
    assert int(st) == sv.SV_ROW_BAD_SLOT
    sv.sv_history_reset(h, n=2)
    want.counts[:2] = 0
    want.prompt[:2] = False
    check_history(h, want)
    sv.sv_history_reset(h)
    check_history(h, plain.History(R, V))


def test_history_from_two_streams_at_once():
    V, R = 2000, 8
    h, want = sv.TokenHistory.empty(R, V, "cuda"), plain.History(R, V)
    rng = np.random.default_rng(5)
    lots = [rng.integers(0, 40, (R, 3000)).astype(np.int32) for _ in range(4)]
    on_gpu = [dev(t) for t in lots]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i, t in enumerate(on_gpu):
        sv.sv_history_add(h, t, stream=streams[i % 2])
    for t in lots:
        for b in range(R):
            want.add(b, t[b])
    check_history(h, want)


# ---------------------------------------------------------------------------
# Rules.
# ---------------------------------------------------------------------------
class Case:
    """A batch with every rule, and its plain result."""

    def __init__(self, B, P, V, dtype, seed, K=None, pos0=0, v0=0, Vs=None, lengths=None, extra=0,
                 n_bias=3, masks="index", penalties=True, slots=False, history=True):
        rng = self.rng = np.random.default_rng(seed)
        self.B, self.P, self.V, self.dtype, self.pos0, self.extra = B, P, V, dtype, pos0, extra
        self.v0, self.Vs = v0, V - v0 if Vs is None else Vs
        K = self.K = P - 1 if K is None else K
        R = B + 3 if slots else B
        z = torch.from_numpy(rng.normal(0, 3, (B, P, V)).astype(np.float32))
        self.z = z.to(DT[dtype])
        self.drafts = rng.integers(0, V, (B, K)).astype(np.int32)
        if K > 1:
            self.drafts[:, 1] = self.drafts[:, 0]                 # a draft twice in a block
        self.lengths = lengths
        self.slots = rng.permutation(R)[:B].astype(np.int32) if slots else None
        self.history = plain.History(R, V)
        if history:
            for s in range(R):
                self.history.add(s, rng.integers(0, V, 3 + V // 20), prompt=True)
                self.history.add(s, rng.integers(0, V, 3 + V // 20))
        self.rep = (1 + rng.random(B)).astype(np.float32) if penalties else np.ones(B, np.float32)
        self.freq = rng.normal(0, 1, B).astype(np.float32) * penalties
        self.pres = rng.normal(0, 1, B).astype(np.float32) * penalties
        self.bias = [dict(zip(rng.permutation(V)[:n_bias].tolist(),
                              rng.normal(0, 3, n_bias).astype(np.float32).tolist()))
                     for _ in range(B)]
        for b in range(B):                                        # biased drafts, a banned token
            if n_bias and K:
                self.bias[b][int(self.drafts[b, 0])] = 1.5
            if n_bias > 1:
                self.bias[b][int(rng.integers(0, V))] = -np.inf
        self.mask = self.index = None
        if masks:
            n = B * P if masks == "all" else 5
            self.mask = rng.random((n, V)) < rng.choice([0.02, 0.5, 0.95, 1.0], (n, 1))
            self.mask[:, rng.integers(0, V, n)] = True
            if masks == "index":
                self.index = rng.integers(-1, n, (B, P)).astype(np.int32)

    def rules(self):
        lists = [list(d.items()) for d in self.bias]
        flat = [e for l in lists for e in l]
        begin = np.cumsum([0] + [len(l) for l in lists]).astype(np.int32)
        h = sv.TokenHistory(self.V, dev(plain.pack(self.history.prompt)),
                            dev(plain.pack(self.history.counts > 0)),
                            dev(self.history.counts.astype(np.int32)))
        return sv.LogitRules(
            h, None if self.slots is None else dev(self.slots), dev(self.rep), dev(self.freq),
            dev(self.pres), dev(begin), dev(np.array([t for t, _ in flat], np.int32)),
            dev(np.array([v for _, v in flat], np.float32)),
            None if self.mask is None else dev(plain.pack(self.mask)),
            None if self.index is None else dev(self.index))

    def n_pos(self, b):
        if self.lengths is None:
            return self.P
        return int(np.clip(int(self.lengths[b]) + self.extra - self.pos0, 0, self.P))

    def want(self):
        z = self.z.double().numpy()
        out, bound = np.empty_like(z), np.empty_like(z)
        for b in range(self.B):
            s = b if self.slots is None else int(self.slots[b])
            masks = [None] * self.P
            if self.mask is not None:
                for p in range(self.P):
                    m = b * self.P + p if self.index is None else self.index[b, p]
                    masks[p] = self.mask[m] if m >= 0 else None
            out[b], bound[b] = plain.process(
                z[b], self.dtype, self.drafts[b], self.pos0, self.n_pos(b),
                self.history.prompt[s], self.history.counts[s], float(self.rep[b]),
                float(self.freq[b]), float(self.pres[b]), self.bias[b], masks)
        cut = slice(self.v0, self.v0 + self.Vs)
        return out[..., cut], bound[..., cut]

    def run(self, in_place, rules=None, shift=0, stream=None):
        """The kernel's result.  The logits stand `shift` elements behind a
        16-byte boundary, the separate output likewise or (shift < 0) at
        another alignment, with guards around both."""
        z = self.z[..., self.v0:self.v0 + self.Vs].contiguous().cuda()
        n, pad = z.numel(), 64

        def place(off, fill):
            buf = torch.full((n + 2 * pad,), fill, dtype=z.dtype, device="cuda")
            return buf, buf[pad + off:pad + off + n].view(z.shape)
        src_buf, src = place(abs(shift), 77.0)
        src.copy_(z)
        out_buf, out = (src_buf, src) if in_place else place(max(shift, 0), 55.0)
        off = abs(shift) if in_place else max(shift, 0)
        if not in_place:
            out.copy_(z.new_full(z.shape, 55.0))
        st = new_status()
        torch.cuda.synchronize()
        sv.sv_logits_process(src, out, rules or self.rules(),
                             dev(self.drafts) if self.K else None,
                             None if self.lengths is None else dev(self.lengths), self.extra,
                             self.pos0, self.V, self.v0, status=st, stream=stream)
        torch.cuda.synchronize()
        fill = 77.0 if in_place else 55.0
        assert bool((out_buf[:pad + off] == fill).all() and (out_buf[pad + off + n:] == fill).all())
        if not in_place:
            assert torch.equal(src.view(torch.uint8), z.view(torch.uint8)), "the input was written"
        return out.cpu().double().numpy(), int(st)

    def check(self, in_place, status=0, want=None, **kw):
        got, st = self.run(in_place, **kw)
        want, bound = want or self.want()
        want = want.copy()
        if not in_place:
            for b in range(self.B):
                want[b, self.n_pos(b):] = 55.0
        plain.check(got, want, bound, f"in_place={in_place} {kw}")
        assert st == status


SIZES = [(1, 1, 1), (1, 1, 5), (2, 3, 31), (2, 2, 32), (3, 2, 33), (4, 5, 1000), (3, 4, 8192),
         (2, 3, 8193), (2, 2, 20011), (1, 65, 300), (5, 9, 777)]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("B,P,V", SIZES)
def test_rules(B, P, V, dtype):
    c = Case(B, P, V, dtype, seed=B + P + V, n_bias=min(3, V))
    want = c.want()
    for in_place in (True, False):
        c.check(in_place, want=want)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("shift", [0, 1, 3, 7, -1, -5])
def test_rules_at_any_alignment(dtype, shift):
    c = Case(3, 4, 8203, dtype, seed=7 + shift, masks="all")
    c.check(False, shift=shift)
    c.check(True, shift=shift)


@pytest.mark.parametrize("kw", [
    dict(masks=None), dict(n_bias=0), dict(penalties=False), dict(history=False), dict(K=0),
    dict(masks=None, n_bias=0, penalties=False), dict(slots=True), dict(n_bias=700),
    dict(K=64, pos0=60), dict(K=3, pos0=3), dict(K=9, pos0=1),
    dict(lengths=[0, -1, 2, 7, 1], extra=1), dict(lengths=[0, -5, 2, 7, 1], extra=0),
    dict(lengths=[3, 4, 5, 6, 9], extra=1, pos0=3, K=8),
], ids=str)
def test_rules_one_by_one(kw):
    kw = dict(kw)
    if "lengths" in kw:
        kw["lengths"] = np.array(kw["lengths"], np.int32)
    for dtype in ("float32", "bfloat16"):
        c = Case(5, 4, 3001, dtype, seed=3, **kw)
        want = c.want()
        for in_place in (True, False):
            c.check(in_place, want=want)


def test_rows_that_share_a_slot():
    c = Case(5, 3, 2000, "bfloat16", seed=29, slots=True)
    c.slots[:] = [4, 1, 4, 4, 1]
    want = c.want()
    for in_place in (True, False):
        c.check(in_place, want=want)


@pytest.mark.parametrize("extra", [0, 1, 2**31 - 1, -2**31])
def test_rules_lengths_at_the_ends_of_their_type(extra):
    lengths = np.array([2**31 - 1, -2**31, 0, 1, -1, 3], np.int64)
    c = Case(6, 4, 700, "float32", seed=31, lengths=lengths.astype(np.int32), extra=extra)
    c.lengths = lengths
    want = c.want()
    c.lengths = lengths.astype(np.int32)
    c.n_pos = lambda b: int(np.clip(int(lengths[b]) + extra, 0, 4))
    for in_place in (True, False):
        c.check(in_place, want=want)


@pytest.mark.parametrize("v0,Vs", [(0, 1), (0, 10001), (5, 8192), (33, 9000), (8191, 1811),
                                   (10001, 1), (64, 64)])
def test_rules_on_a_vocabulary_slice(v0, Vs):
    c = Case(3, 3, 10002, "bfloat16", seed=v0, v0=v0, Vs=Vs)
    want = c.want()
    for in_place in (True, False):
        c.check(in_place, want=want)


def test_rules_large_vocabulary():
    c = Case(2, 2, 1 << 20, "bfloat16", seed=1, n_bias=50)
    want = c.want()
    for in_place in (True, False):
        c.check(in_place, want=want)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_masked_infinities_and_nans(dtype):
    """A forbidden logit is -inf whatever it was; an allowed one keeps what
    arithmetic makes of it; the type's lowest value is an ordinary logit."""
    c = Case(2, 3, 400, dtype, seed=11, n_bias=0, masks="all")
    lowest = torch.finfo(DT[dtype]).min
    for i, v in enumerate([np.inf, -np.inf, np.nan, lowest]):
        c.z[..., i::9] = v
    c.rep[:] = 1.0                     # the lowest value times a repetition would leave the range
    c.freq[:] = c.pres[:] = 0.25
    for in_place in (True, False):
        c.check(in_place)


def test_empty_masks_leave_only_minus_infinity():
    c = Case(3, 2, 9001, "bfloat16", seed=13, masks="all")
    c.mask[2 * 1 + 1] = False          # row 1, position 1
    for in_place in (True, False):
        got, st = c.run(in_place)
        assert np.all(got[1, 1] == -np.inf) and st == sv.SV_ROW_EMPTY_MASK
        c.check(in_place, status=sv.SV_ROW_EMPTY_MASK)
    # allowed bits behind the vocabulary's end allow nothing
    words = plain.pack(c.mask)
    words[3, -1] = np.int32(-1) << (9001 % 32)
    r = c.rules()
    r2 = sv.LogitRules(mask=dev(words))
    c.bias = [{} for _ in c.bias]
    c.rep[:], c.freq[:], c.pres[:] = 1, 0, 0
    c.check(True, status=sv.SV_ROW_EMPTY_MASK, rules=r2)
    del r


def test_last_entry_of_a_token_listed_twice_counts():
    V, B = 9000, 2
    c = Case(B, 3, V, "float32", seed=17, n_bias=0, masks=None)
    tokens = np.array([5, 8999, 5, 8999, 5, 7, 5, 6, 6], np.int32)
    values = np.array([1, 2, 3, -np.inf, 4, 5, np.nan, 6, np.inf], np.float32)
    begin = np.array([0, 7, 9], np.int32)
    c.bias = [{5: 4.0, 8999: -np.inf, 7: 5.0}, {6: 6.0}]     # NaN and +inf are left out
    base = c.rules()
    r = sv.LogitRules(base.history, repetition=dev(c.rep), frequency=dev(c.freq),
                      presence=dev(c.pres), bias_begin=dev(begin), bias_tokens=dev(tokens),
                      bias_values=dev(values))
    for in_place in (True, False):
        c.check(in_place, rules=r, status=sv.SV_ROW_BAD_BIAS)


def test_bad_data_is_left_out_and_reported():
    c = Case(6, 3, 500, "float32", seed=19, masks="index", slots=True)
    c.rep[0], c.rep[1], c.rep[2] = np.nan, 0.0, -1.0
    c.freq[3], c.pres[4], c.rep[5] = np.inf, np.nan, np.inf
    c.index[2, 1], c.index[3, 0] = 5, -2
    c.drafts[1, 0], c.drafts[2, 0] = -1, 500
    c.bias[1] = c.bias[2] = {}
    for b in (1, 2):
        c.drafts[b, 1] = 3
    c.slots[5] = 99
    rules = c.rules()
    r = rules.desc
    bits = (sv.SV_ROW_BAD_PENALTY | sv.SV_ROW_BAD_MASK | sv.SV_ROW_BAD_TOKEN | sv.SV_ROW_BAD_SLOT)
    c.rep[[0, 1, 2, 5]], c.freq[3], c.pres[4] = 1.0, 0.0, 0.0
    c.index[2, 1] = c.index[3, 0] = -1
    c.slots[5] = c.history.counts.shape[0]
    c.history.counts = np.vstack([c.history.counts, np.zeros((1, 500), np.int64)])
    c.history.prompt = np.vstack([c.history.prompt, np.zeros((1, 500), bool)])
    want = c.want()
    for in_place in (True, False):
        c.check(in_place, rules=rules, status=bits, want=want)
    del r
    # a bias list outside its arrays, a token outside the vocabulary
    c = Case(3, 1, 500, "float32", seed=23, masks=None, n_bias=0)
    base = c.rules()
    for begin, tokens, bias, bits in (
            ([0, 1, 3, 9], [4, 5, 6], [{4: 1.0}, {5: 1.0, 6: 1.0}, {}], sv.SV_ROW_BAD_BIAS),
            ([0, 2, 1, 1], [4, 5, 6], [{4: 1.0, 5: 1.0}, {}, {}], sv.SV_ROW_BAD_BIAS),
            ([-1, 1, 2, 3], [4, 500, -7], [{}, {}, {}], sv.SV_ROW_BAD_BIAS | sv.SV_ROW_BAD_TOKEN)):
        c.bias = bias
        rules = sv.LogitRules(base.history, repetition=dev(c.rep), frequency=dev(c.freq),
                              presence=dev(c.pres), bias_begin=dev(np.array(begin, np.int32)),
                              bias_tokens=dev(np.array(tokens, np.int32)),
                              bias_values=dev(np.ones(3, np.float32)))
        c.check(True, rules=rules, status=bits)


def test_rules_behind_four_gigabytes():
    """Rows whose logits lie more than 2^32 bytes behind the first one."""
    B, P, V = 1060, 16, 129280                  # 2.19e9 elements
    z = torch.zeros(B, P, V, dtype=torch.bfloat16, device="cuda")
    z[-1] = 2.0
    z[0] = 2.0
    lengths = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    lengths[0] = lengths[-1] = P
    mask = torch.full((1, (V + 31) // 32), -1, dtype=torch.int32, device="cuda")
    mask[0, 7] = 0
    index = torch.zeros(B, P, dtype=torch.int32, device="cuda")
    drafts = torch.full((B, P - 1), V - 1, dtype=torch.int32, device="cuda")
    rules = sv.LogitRules(frequency=torch.full((B,), 0.5, device="cuda"), mask=mask,
                          mask_index=index)
    sv.sv_logits_process(z, z, rules, drafts, lengths)
    want = torch.full((P, V), 2.0, dtype=torch.bfloat16, device="cuda")
    want[:, 7 * 32:8 * 32] = -float("inf")
    want[:, -1] -= 0.5 * torch.arange(P, device="cuda")
    assert torch.equal(z[0], want) and torch.equal(z[-1], want)
    assert not bool(z[1:-1].any())


def test_rules_on_streams_and_in_a_graph():
    cases = [Case(4, 5, 5000, "bfloat16", seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in cases]
    for c, s in zip(cases, streams):
        c.check(True, stream=s)
    # both at once, then captured and replayed on fresh logits
    z = [c.z.cuda() for c in cases]
    rules, drafts = [c.rules() for c in cases], [dev(c.drafts) for c in cases]
    want = [c.want() for c in cases]
    torch.cuda.synchronize()
    for i, s in enumerate(streams):
        sv.sv_logits_process(z[i], z[i], rules[i], drafts[i], stream=s)
    torch.cuda.synchronize()
    for i in range(2):
        plain.check(z[i].cpu().double().numpy(), *want[i])
    graph = torch.cuda.CUDAGraph()
    out = torch.zeros_like(z[0])
    with torch.cuda.graph(graph):
        sv.sv_logits_process(z[0], out, rules[0], drafts[0])
        sv.sv_logits_process(z[1], z[1], rules[1], drafts[1])
    for _ in range(2):
        for i in range(2):
            z[i].copy_(cases[i].z)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        plain.check(out.cpu().double().numpy(), *want[0])
        plain.check(z[1].cpu().double().numpy(), *want[1])


@pytest.mark.parametrize("n_more", [0, 300])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_a_bias_of_minus_infinity_bans_whatever_the_logit_was(dtype, n_more):
    """n_more further biases in the chunk: none, and more than a CTA lists."""
    V = 2000
    c = Case(2, 3, V, dtype, seed=37, n_bias=0, masks=None)
    c.bias = [{}, {}]
    c.rep[:] = 1.0
    c.freq[:] = c.pres[:] = 0.25
    for i, v in enumerate([np.inf, np.nan, -np.inf, torch.finfo(DT[dtype]).min]):
        c.z[..., i::9] = v
    banned = np.arange(0, 40)
    for b in range(2):
        c.bias[b] = {int(t): -np.inf for t in banned}
        c.bias[b].update({1000 + t: 0.5 for t in range(n_more)})
    want, bound = c.want()
    want[..., banned], bound[..., banned] = -np.inf, 0.0
    for in_place in (True, False):
        c.check(in_place, want=(want, bound))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n", [255, 256, 257, 700, 5000])
def test_tokens_listed_again_in_long_lists(n, dtype):
    """Lists around and past what a CTA keeps on chip, half of their tokens listed
    again: the last valid entry counts, whatever chunk it lies in."""
    V, B = 20011, 2
    c = Case(B, 3, V, dtype, seed=41 + n, n_bias=0)
    tokens, values, c.bias = [], [], []
    for b in range(B):
        few = c.rng.integers(0, 8192 if b else V, n // 2)   # row 1: all in one chunk in place
        t = np.concatenate([few, c.rng.choice(few, n - n // 2)]).astype(np.int32)
        v = c.rng.normal(0, 3, n).astype(np.float32)
        v[c.rng.random(n) < 0.2] = -np.inf
        v[c.rng.random(n) < 0.2] = np.nan
        v[c.rng.random(n) < 0.1] = np.inf
        c.bias.append({int(x): float(y) for x, y in zip(t, v) if y < np.inf})   # NaN: false
        tokens.append(t)
        values.append(v)
    base = c.rules()
    r = sv.LogitRules(base.history, repetition=dev(c.rep), frequency=dev(c.freq),
                      presence=dev(c.pres), bias_begin=dev(np.array([0, n, 2 * n], np.int32)),
                      bias_tokens=dev(np.concatenate(tokens)),
                      bias_values=dev(np.concatenate(values)),
                      mask=dev(plain.pack(c.mask)), mask_index=dev(c.index))
    want = c.want()
    for in_place in (True, False):
        c.check(in_place, rules=r, status=sv.SV_ROW_BAD_BIAS, want=want)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("near,far", [(8192, 0), (200, 60000)])
def test_one_repeated_bias_does_not_cost_more_than_its_entry(near, far, in_place):
    """The same list with and without one repeated token.  Each entry is read
    once or twice either way, so the times are alike (a factor of three is
    left for noise); a scan of the list for each entry would make them differ
    by the list's length."""
    V, P = 129280, 9
    z = torch.zeros(1, P, V, device="cuda")
    out = z if in_place else torch.zeros_like(z)
    took = []
    for repeat in (False, True):
        tokens = np.concatenate([np.arange(near), 20000 + np.arange(far)]).astype(np.int32)
        if repeat:
            tokens[1] = tokens[0]
        rules = sv.LogitRules(bias_begin=dev(np.array([0, near + far], np.int32)),
                              bias_tokens=dev(tokens),
                              bias_values=torch.full((near + far,), 1.0, device="cuda"))
        times = []
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            sv.sv_logits_process(z, out, rules)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        took.append(min(times))
    assert took[1] <= 3 * took[0] + 0.05, f"{took[0]:.3f} ms without, {took[1]:.3f} ms with"


def test_a_bias_list_over_empty_arrays_is_reported():
    c = Case(2, 2, 300, "float32", seed=43, n_bias=0, masks=None)
    c.bias = [{}, {}]
    base = c.rules()
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    for begin, bits in (([0, 0, 0], 0), ([0, 0, 5], sv.SV_ROW_BAD_BIAS)):
        r = sv.LogitRules(base.history, repetition=dev(c.rep), frequency=dev(c.freq),
                          presence=dev(c.pres), bias_begin=dev(np.array(begin, np.int32)),
                          bias_tokens=none, bias_values=none.float())
        for in_place in (True, False):
            c.check(in_place, rules=r, status=bits)


def test_history_of_more_entries_than_threads():
    """The kernels start at most 148 * 64 * 256 = 2424832 threads."""
    B, S, V = 300, 9001, 1000
    tokens = torch.randint(0, V, (B, S), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    h = sv.TokenHistory.empty(B, V, "cuda")
    for kind in (sv.SV_HISTORY_PROMPT, sv.SV_HISTORY_OUTPUT):
        sv.sv_history_add(h, tokens.cuda(), kind=kind)
    counts = torch.zeros(B, V, dtype=torch.int32).scatter_add_(
        1, tokens.long(), torch.ones_like(tokens)).numpy()
    assert np.array_equal(h.output_counts.cpu().numpy(), counts)
    for bits in (h.output_bits, h.prompt_bits):
        assert np.array_equal(bits.cpu().numpy(), plain.pack(counts > 0))
    R = 2500000                                  # slots of one word each
    h = sv.TokenHistory.empty(R, 3, "cuda")
    h.prompt_bits.fill_(5)
    h.output_bits.fill_(6)
    h.output_counts[:, 1:] = 7
    sv.sv_history_reset(h, n=R - 1)
    for t, last in ((h.prompt_bits, [5]), (h.output_bits, [6]), (h.output_counts, [0, 7, 7])):
        assert not bool(t[:-1].any()) and t[-1].tolist() == last


@pytest.mark.parametrize("v0,Vs", [(0, 10001), (5, 8192), (33, 9000), (8191, 1811), (10001, 1)])
def test_rules_on_a_vocabulary_slice_in_fp32(v0, Vs):
    c = Case(3, 3, 10002, "float32", seed=v0 + 1, v0=v0, Vs=Vs, slots=True)
    want = c.want()
    for in_place in (True, False):
        c.check(in_place, want=want)


@pytest.mark.parametrize("seed", range(60))
def test_rules_of_random_batches(seed):
    rng = np.random.default_rng(1000 + seed)
    V = int(np.exp(rng.uniform(0, np.log(30000))))
    P = int(rng.choice([1, 1, 2, 3, 5, 9, 17, 65]))
    B = max(1, min(int(np.exp(rng.uniform(0, np.log(40)))), 300000 // (P * V)))
    K = min(64, int(rng.choice([0, P - 1, P, P + 3])))
    v0 = int(rng.choice([0, 0, rng.integers(0, V)]))
    lengths = rng.integers(-2, P + 3, B).astype(np.int32) if rng.random() < 0.5 else None
    c = Case(B, P, V, str(rng.choice(["float32", "bfloat16"])), seed=seed, K=K,
             pos0=int(rng.choice([0, 0, rng.integers(0, 6)])), v0=v0,
             Vs=int(rng.choice([V - v0, rng.integers(1, V - v0 + 1)])), lengths=lengths,
             extra=int(rng.integers(0, 3)), n_bias=int(min(V, rng.choice([0, 1, 3, 16, 400]))),
             masks=[None, "index", "all"][rng.integers(0, 3)], penalties=bool(rng.random() < 0.8),
             slots=bool(rng.random() < 0.5), history=bool(rng.random() < 0.8))
    want = c.want()
    for in_place in (True, False):
        c.check(in_place, want=want, shift=int(rng.integers(-9, 10)))


def test_history_behind_four_gigabytes():
    """Slots whose counts lie more than 2^32 elements behind the first one's."""
    R, V = 34000, 129280                          # 4.4e9 counts
    h = sv.TokenHistory.empty(R, V, "cuda")
    slots = np.array([0, 16612, 33222, R - 1], np.int32)
    rng = np.random.default_rng(3)
    tokens = rng.integers(0, V, (4, 50)).astype(np.int32)
    for kind in (sv.SV_HISTORY_PROMPT, sv.SV_HISTORY_OUTPUT):
        sv.sv_history_add(h, dev(tokens), kind=kind, slots=dev(slots))
    counts = np.zeros((4, V), np.int32)
    for b in range(4):
        np.add.at(counts[b], tokens[b], 1)
    at = dev(slots).long()
    assert np.array_equal(h.output_counts[at].cpu().numpy(), counts)
    assert np.array_equal(h.prompt_bits[at].cpu().numpy(), plain.pack(counts > 0))
    for in_place in (True, False):
        z = torch.full((4, 1, V), 2.0, device="cuda")
        out = z if in_place else torch.zeros_like(z)
        sv.sv_logits_process(z, out, sv.LogitRules(h, dev(slots), frequency=torch.full((4,), 0.5, device="cuda")))
        assert np.array_equal(out[:, 0].cpu().numpy(), 2.0 - 0.5 * counts.astype(np.float32))
    assert int(h.output_counts.sum(1, dtype=torch.int32).sum()) == 200
    sv.sv_history_reset(h, dev(slots[1:]))
    assert int(h.output_counts.sum(1, dtype=torch.int32).sum()) == 50
    assert np.array_equal(h.output_counts[0].cpu().numpy(), counts[0])
    assert not bool(h.prompt_bits[at[1:]].any() or h.output_bits[at[1:]].any())


def test_history_in_a_graph():
    V, B = 500, 3
    h, want = sv.TokenHistory.empty(B, V, "cuda"), plain.History(B, V)
    rng = np.random.default_rng(4)
    tokens = torch.zeros(B, 6, dtype=torch.int32, device="cuda")
    one = dev(np.array([1], np.int32))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.sv_history_reset(h, one)
        sv.sv_history_add(h, tokens)
        sv.sv_history_add(h, tokens, kind=sv.SV_HISTORY_PROMPT)
    for _ in range(3):
        t = rng.integers(0, V, (B, 6)).astype(np.int32)
        tokens.copy_(dev(t))
        graph.replay()
        want.counts[1], want.prompt[1] = 0, False
        for b in range(B):
            want.add(b, t[b])
            want.add(b, t[b], prompt=True)
        check_history(h, want)
