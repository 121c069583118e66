"""The 4-bit output head on the GPU against its plain 64-bit form, and the
chain head -> rules -> verification -> history."""
import threading

import numpy as np
import pytest
import torch

import _plain_rules as plain
import speculative_decoding_verification_93_b200 as sv
from oracle import compare as ocompare

pytestmark = pytest.mark.gpu

DT = {"float32": torch.float32, "bfloat16": torch.bfloat16}


class Head:
    def __init__(self, H, V, group, zero, scale, seed):
        rng = self.rng = np.random.default_rng(seed)
        G = H // group
        self.H, self.V, self.group = H, V, group
        self.codes = rng.integers(0, 16, (V, H)).astype(np.uint8)
        self.zero = rng.integers(0, 16, (V, G)).astype(np.uint8) if zero else None
        self.scale = torch.from_numpy(rng.uniform(0.01, 0.1, (V, G)).astype(np.float32)).to(DT[scale])
        packed = torch.from_numpy(self.codes[:, 0::2] | self.codes[:, 1::2] << 4).cuda()
        # the high half of a zero's byte is not part of it
        z = None if self.zero is None else torch.from_numpy(self.zero | 0xa0).cuda()
        self.weight = sv.W4Weight(packed, self.scale.cuda(), z)

    def want(self, x, dtype):
        zero = self.zero if self.zero is not None else np.full(self.scale.shape, 8)
        out, bound = plain.head(x.double().cpu().numpy().reshape(-1, self.H), self.codes,
                                self.scale.double().numpy(), zero, self.group, dtype)
        return out.reshape(*x.shape[:2], self.V), bound.reshape(*x.shape[:2], self.V)

    def run(self, x, dtype, lengths=None, extra=0, stream=None):
        B, P, _ = x.shape
        n, pad = B * P * self.V, 64
        buf = torch.full((n + 2 * pad,), 55.0, dtype=DT[dtype], device="cuda")
        out = buf[pad + 1:pad + 1 + n].view(B, P, self.V)      # no 16-byte boundary
        need = sv.sv_head_w4_workspace_bytes(self.weight, B, P)
        ws = torch.full((need + 16,), 255, dtype=torch.uint8, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        sv.sv_head_w4(self.weight, x, out, ws[:need] if need else None, lengths=lengths,
                      extra=extra, status=st, stream=stream)
        torch.cuda.synchronize()
        assert bool((buf[:pad + 1] == 55).all() and (buf[pad + 1 + n:] == 55).all())
        assert bool((ws[need:] == 255).all()) and int(st) == 0
        return out

    def check(self, x, dtype, lengths=None, extra=0, **kw):
        got = self.run(x, dtype, lengths, extra, **kw).double().cpu().numpy()
        want, bound = self.want(x, dtype)
        if lengths is not None:
            for b, n in enumerate(lengths.tolist()):
                want[b, max(0, n + extra):], bound[b, max(0, n + extra):] = 55.0, 0.0
        plain.check(got, want, bound)

    def x(self, B, P):
        return torch.from_numpy(self.rng.normal(0, 1, (B, P, self.H)).astype(np.float32)).to(
            "cuda", torch.bfloat16)


SHAPES = [(32, 1, 32), (64, 7, 32), (64, 8, 64), (128, 33, 128), (96, 100, 32), (256, 129, 64),
          (1120, 1000, 32), (4096, 257, 128), (2048 + 64, 300, 64), (1408, 515, 128)]


@pytest.mark.parametrize("H,V,group", SHAPES)
@pytest.mark.parametrize("zero,scale", [(False, "bfloat16"), (True, "float32")])
def test_head(H, V, group, zero, scale):
    h = Head(H, V, group, zero, scale, seed=H + V)
    for B, P in ((1, 1), (1, 2), (3, 1), (1, 5), (1, 8), (3, 3), (2, 8), (1, 9), (17, 1)):
        for dtype in ("float32", "bfloat16"):
            h.check(h.x(B, P), dtype)


@pytest.mark.parametrize("M", [24, 31, 32, 33, 48, 63, 64, 65, 80, 96, 127, 128, 129, 255, 256, 257, 320,
                               600])
@pytest.mark.parametrize("H,V,group,zero", [(256, 300, 64, False), (1120, 131, 32, True),
                                            (1024, 260, 128, True)])
def test_head_many_tokens(M, H, V, group, zero):
    h = Head(H, V, group, zero, "bfloat16", seed=M)
    for dtype in ("float32", "bfloat16"):
        h.check(h.x(M, 1), dtype)


@pytest.mark.parametrize("H,M", [(16384, 1), (16384, 9), (32768, 1), (32768, 3), (12160, 8), (12288, 16)])
def test_head_long_rows(H, M):
    h = Head(H, 150, 64, True, "bfloat16", seed=H + M)
    for dtype in ("float32", "bfloat16"):
        h.check(h.x(M, 1), dtype)


@pytest.mark.parametrize("V", [16 * 4 * 148, 16 * 4 * 148 + 1, 40000])
def test_head_few_tokens_of_a_large_vocabulary(V):
    h = Head(160, V, 32, True, "bfloat16", seed=V)
    for M in (1, 8, 16):
        h.check(h.x(M, 1), "float32")


@pytest.mark.parametrize("M", [20, 50, 100, 200, 1030])
@pytest.mark.parametrize("H,V,group,zero", [(4608, 1000, 128, False), (2112, 701, 64, True), (1600, 515, 32, True),
                                            (12288, 129, 128, True), (4096, 9000, 64, False), (2048, 1, 32, False)])
def test_head_long_rows_of_a_small_vocabulary(M, H, V, group, zero):
    # few tiles: several blocks share each tile's k
    h = Head(H, V, group, zero, "float32" if zero else "bfloat16", seed=M + H)
    P = 5 if M % 5 == 0 else 1
    x = h.x(M // P, P)
    lengths = torch.from_numpy(h.rng.integers(-1, P + 1, M // P).astype(np.int32)).cuda()
    for out in ("float32", "bfloat16"):
        h.check(x, out)
        h.check(x, out, lengths, 1)
    assert torch.equal(h.run(x, "float32"), h.run(x, "float32"))


# Blocks of 128 k of a warp's share: 1, 2, 3, 5, 9 and unequal ones, four (the
# large vocabulary) or sixteen warps to a tile, several tiles a warp.
@pytest.mark.parametrize("V,H", [(40000, 512), (40000, 640), (40000, 1536), (40000, 2112), (40000, 2560), (40000, 4608),
                                 (6000, 2048), (6000, 4160), (6000, 6144), (6000, 10240)])
@pytest.mark.parametrize("group,zero,scale", [(128, False, "bfloat16"), (64, True, "float32"), (32, True, "bfloat16")])
def test_head_few_tokens_whatever_a_warps_share(V, H, group, zero, scale):
    h = Head(H // group * group, V, group, zero, scale, seed=V + H)
    for M in (2, 10):
        h.check(h.x(M, 1), "float32")


@pytest.mark.parametrize("M", [17, 40, 64, 100, 200])
@pytest.mark.parametrize("H,group,zero", [(384, 128, False), (128, 128, True), (96, 32, True), (448, 64, False),
                                          (1120, 32, True), (2112, 64, True), (1408, 128, False)])
def test_head_several_tiles_a_block(M, H, group, zero):
    # three tiles of 128 rows for some blocks; odd and even numbers of groups
    h = Head(H, 2 * 148 * 128 + 130, group, zero, "bfloat16", seed=M + H)
    h.check(h.x(M, 1), "bfloat16")


@pytest.mark.parametrize("B,P", [(1, 1), (5, 4), (40, 5), (3, 9), (16, 1)])
def test_head_leaves_unscheduled_positions_as_they_were(B, P):
    h = Head(512, 1031, 128, True, "bfloat16", seed=B)
    for extra in (0, 1):
        lengths = torch.from_numpy(h.rng.integers(-2, P + 2, B).astype(np.int32)).cuda()
        x = h.x(B, P)
        for b, n in enumerate(lengths.tolist()):
            x[b, max(0, n + extra):] = float("nan")            # never read into another row
        h.check(x, "bfloat16", lengths, extra)
        none = torch.full((B,), -1, dtype=torch.int32, device="cuda")
        h.check(x, "float32", none, extra)


@pytest.mark.parametrize("M", [3, 9, 40, 130])
def test_head_infinities_stay_in_their_row(M):
    h = Head(256, 140, 64, False, "float32", seed=M)
    x = h.x(M, 1)
    x[1, 0, 5], x[2, 0, 250] = float("inf"), float("nan")
    got = h.run(x, "float32").double().cpu().numpy()
    want, bound = h.want(x.nan_to_num(0, 0, 0), "float32")
    clean = [t for t in range(M) if t not in (1, 2)]
    plain.check(got[clean], want[clean], bound[clean])
    assert np.isnan(got[2]).all() and not np.isfinite(got[1]).any()


def test_head_same_bits_every_time():
    h = Head(1024, 700, 128, False, "bfloat16", seed=3)
    for M in (1, 9, 70):
        x = h.x(M, 1)
        first = h.run(x, "float32")
        for _ in range(3):
            assert torch.equal(h.run(x, "float32"), first)


def test_head_on_streams_and_in_a_graph():
    h = Head(512, 2000, 64, True, "bfloat16", seed=9)
    for M in (1, 20, 140):
        xs = [h.x(M, 1) for _ in range(2)]
        want = [h.want(x, "float32") for x in xs]
        outs = [torch.zeros(M, 1, 2000, device="cuda") for _ in xs]
        need = sv.sv_head_w4_workspace_bytes(h.weight, M, 1)
        ws = [torch.empty(max(need, 16), dtype=torch.uint8, device="cuda") for _ in xs]
        streams = [torch.cuda.Stream() for _ in xs]
        torch.cuda.synchronize()
        for i, s in enumerate(streams):
            sv.sv_head_w4(h.weight, xs[i], outs[i], ws[i], stream=s)
        torch.cuda.synchronize()
        for i in range(2):
            plain.check(outs[i].double().cpu().numpy(), *want[i])
        # two graphs that share a workspace, replayed one after the other
        graphs = []
        for i in range(2):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[i]):
                sv.sv_head_w4(h.weight, xs[i], outs[i], ws[0])
        for _ in range(2):
            for o in outs:
                o.zero_()
            for g in graphs:
                g.replay()
            torch.cuda.synchronize()
            for i in range(2):
                plain.check(outs[i].double().cpu().numpy(), *want[i])


@pytest.mark.parametrize("M", [1, 20, 140])
def test_head_of_a_small_vocabulary_replayed(M):
    # a graph whose input changes between replays, beside eager calls on another stream
    h = Head(4608, 1000, 128, True, "bfloat16", seed=M)
    xs = [h.x(M, 1) for _ in range(3)]
    want = [h.want(x, "float32") for x in xs]
    x, outs = xs[0].clone(), [torch.zeros(M, 1, 1000, device="cuda") for _ in range(2)]
    need = sv.sv_head_w4_workspace_bytes(h.weight, M, 1)
    ws = [torch.empty(max(need, 16), dtype=torch.uint8, device="cuda") for _ in range(2)]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        sv.sv_head_w4(h.weight, x, outs[0], ws[0])
    for i in range(3):
        x.copy_(xs[i])
        torch.cuda.synchronize()
        graph.replay()
        sv.sv_head_w4(h.weight, xs[2], outs[1], ws[1], stream=side)
        torch.cuda.synchronize()
        plain.check(outs[0].double().cpu().numpy(), *want[i])
        plain.check(outs[1].double().cpu().numpy(), *want[2])
        for o in outs:
            o.zero_()


def test_head_from_two_host_threads():
    # threads that have made no CUDA call before, one stream each
    h = Head(512, 2000, 64, True, "bfloat16", seed=13)
    for M in (9, 20, 140):
        xs = [h.x(M, 1) for _ in range(2)]
        outs = [torch.zeros(M, 1, 2000, device="cuda") for _ in xs]
        need = sv.sv_head_w4_workspace_bytes(h.weight, M, 1)
        ws = [torch.empty(max(need, 16), dtype=torch.uint8, device="cuda") for _ in xs]
        streams = [torch.cuda.Stream().cuda_stream for _ in xs]
        torch.cuda.synchronize()
        failed = []

        def call(i):
            try:
                for _ in range(5):
                    sv.sv_head_w4(h.weight, xs[i], outs[i], ws[i], stream=streams[i])
            except Exception as e:
                failed.append(e)

        threads = [threading.Thread(target=call, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        assert not failed
        for i in range(2):
            plain.check(outs[i].double().cpu().numpy(), *h.want(xs[i], "float32"))


@pytest.mark.parametrize("B,P", [(6, 2), (30, 3)])
def test_head_lengths_at_the_ends_of_their_type(B, P):
    h = Head(128, 100, 32, False, "float32", seed=17)
    x, ends = h.x(B, P), torch.tensor([2**31 - 1, -2**31, 0, 1, -1, P], dtype=torch.int32)
    lengths = ends.repeat(B // 6).cuda()
    for extra in (0, 1, 2**31 - 1, -2**31):
        want, bound = h.want(x, "float32")
        for b, n in enumerate(lengths.tolist()):
            want[b, max(0, n + extra):], bound[b, max(0, n + extra):] = 55.0, 0.0
        got = h.run(x, "float32", lengths, extra).double().cpu().numpy()
        plain.check(got, want, bound)


def test_head_most_tokens():
    # 2^20 positions, the most of a call, and one fewer scheduled
    h = Head(32, 33, 32, False, "float32", seed=19)
    x = torch.randint(-3, 4, (1 << 17, 8, 32), dtype=torch.int8, device="cuda").bfloat16()
    lengths = torch.full((1 << 17,), 8, dtype=torch.int32, device="cuda")
    lengths[5] = 7
    got = h.run(x, "float32", lengths)
    w = torch.from_numpy((h.codes.astype(np.float64) - 8)).cuda() * h.scale.double().cuda()
    want = x.double() @ w.T
    # integers of at most 32 * 3 * 8 are exact; the scale's product rounds once
    bound = want.abs() * 2.0 ** -24
    want[5, 7], bound[5, 7] = 55.0, 0.0
    assert bool(((got.double() - want).abs() <= bound).all())


def test_head_refuses_a_short_workspace():
    h = Head(4096, 1000, 128, False, "bfloat16", seed=1)
    for M in (1, 100):
        need = sv.sv_head_w4_workspace_bytes(h.weight, M, 1)
        if need == 0:
            continue
        x, out = h.x(M, 1), torch.zeros(M, 1, 1000, device="cuda")
        with pytest.raises(sv.SVError) as e:
            sv.sv_head_w4(h.weight, x, out, torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
        assert e.value.code == 4


@pytest.mark.parametrize("B,K,V,seed", [(4, 4, 1000, 0), (9, 3, 2051, 1), (64, 5, 1500, 2)])
def test_head_rules_verification_and_history_together(B, K, V, seed):
    """Two decoding steps of a small model: the target's and the drafter's
    heads, the rules of every request, verification, and the history that
    the second step's penalties read.  Verification is checked against the
    oracle on the processed logits themselves."""
    rng = np.random.default_rng(seed)
    target, drafter = Head(256, V, 64, True, "bfloat16", seed), Head(128, V, 32, False, "float32", seed + 1)
    history, plain_history = sv.TokenHistory.empty(B, V, "cuda"), plain.History(B, V)
    dev = lambda x: torch.as_tensor(np.ascontiguousarray(x)).cuda()  # noqa: E731
    rep, freq, pres = (rng.uniform(lo, hi, B).astype(np.float32)
                       for lo, hi in ((1.0, 1.5), (0, 0.4), (0, 0.4)))
    ban = rng.integers(0, V, B).astype(np.int32)
    temp = rng.choice([0.0, 0.7, 1.0], B).astype(np.float32)
    prompt = rng.integers(0, V, (B, 30)).astype(np.int32)
    sv.sv_history_add(history, dev(prompt), kind=sv.SV_HISTORY_PROMPT)
    for b in range(B):
        plain_history.add(b, prompt[b], prompt=True)
    for step in range(2):
        allowed = rng.random((B, K + 1, V)) < np.where(np.arange(B) % 3 == 0, 0.3, 1.0)[:, None, None]
        drafts = rng.integers(0, V, (B, K)).astype(np.int32)
        drafts[1 % B] = drafts[1 % B, 0]
        for i in range(K):                     # drafts come from the grammar
            allowed[np.arange(B), i, drafts[:, i]] = True
        lengths = rng.integers(0, K + 1, B).astype(np.int32)
        rules = dict(history=history, repetition=dev(rep), frequency=dev(freq), presence=dev(pres),
                     bias_begin=dev(np.arange(B + 1, dtype=np.int32)), bias_tokens=dev(ban),
                     bias_values=dev(np.full(B, -3.0, np.float32)))
        words = plain.pack(allowed)
        on_target = sv.LogitRules(**rules, mask=dev(words.reshape(B * (K + 1), -1)))
        on_draft = sv.LogitRules(**rules, mask=dev(words[:, :K].reshape(B * K, -1)))
        xt, xd = target.x(B, K + 1), drafter.x(B, K)
        ln, dr = dev(lengths), dev(drafts)
        zt = torch.full((B, K + 1, V), 9.0, device="cuda")
        zd = torch.full((B, K, V), 9.0, device="cuda")
        ws = torch.empty(max(16, sv.sv_head_w4_workspace_bytes(target.weight, B, K + 1),
                             sv.sv_head_w4_workspace_bytes(drafter.weight, B, K)),
                         dtype=torch.uint8, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        sv.sv_head_w4(target.weight, xt, zt, ws, lengths=ln, extra=1)
        sv.sv_head_w4(drafter.weight, xd, zd, ws, lengths=ln)
        raw = zt.clone(), zd.clone()
        sv.sv_logits_process(zt, zt, on_target, dr, ln, extra=1, status=st)
        sv.sv_logits_process(zd, zd, on_draft, dr, ln, status=st)
        tokens, accepted = sv.verify(zt, zd, dr, ln, dev(temp), seed=77 + step, status=st)
        sv.sv_history_add(history, tokens, accepted, extra=1, status=st)
        torch.cuda.synchronize()
        assert int(st) & ~(sv.SV_NOTE_CDF_FALLBACK | sv.SV_NOTE_ZERO_RESIDUAL) == 0
        bias = [{int(t): -3.0} for t in ban]
        for b in range(B):                     # the logits that verification saw
            for z, before, extra in ((zt, raw[0], 1), (zd, raw[1], 0)):
                n = int(lengths[b]) + extra
                if n == 0:
                    continue
                want, bound = plain.process(
                    before[b].double().cpu().numpy(), "float32", drafts[b], 0, n,
                    plain_history.prompt[b], plain_history.counts[b], float(rep[b]), float(freq[b]),
                    float(pres[b]), bias[b], list(allowed[b]))
                plain.check(z[b].double().cpu().numpy(), want, bound)
        zt_h, zd_h = zt.cpu().numpy(), zd.cpu().numpy()
        tally = ocompare.check_rows(lambda idx: (zt_h[idx], zd_h[idx]), drafts, temp, 77 + step,
                                    lengths, lengths, lengths, lengths, tokens.cpu().numpy(),
                                    accepted.cpu().numpy())
        assert tally.invalid == 0, tally.first_invalid
        tok, acc = tokens.cpu().numpy(), accepted.cpu().numpy()
        for b in range(B):
            emitted = tok[b, :acc[b] + 1]
            assert all(allowed[b, i, t] for i, t in enumerate(emitted))
            plain_history.add(b, emitted)
        assert np.array_equal(history.output_counts.cpu().numpy(), plain_history.counts)
        assert np.array_equal(history.output_bits.cpu().numpy(), plain.pack(plain_history.counts > 0))


def test_head_one_workspace_for_every_batch():
    # 1000 rows: the shares of k have sums in the workspace up to 1024 tokens
    h = Head(2048, 1000, 128, False, "bfloat16", seed=23)
    most = 1100
    ws = torch.empty(sv.sv_head_w4_workspace_bytes(h.weight, most, 1), dtype=torch.uint8, device="cuda")
    for M in (most, 1024, 300, 40, 7):
        x, out = h.x(M, 1), torch.zeros(M, 1, 1000, device="cuda")
        sv.sv_head_w4(h.weight, x, out, ws)
        torch.cuda.synchronize()
        plain.check(out.double().cpu().numpy(), *h.want(x, "float32"))


def test_chain_with_slots_and_one_status():
    """The serving loop as documented: rows mapped to slots, one status word
    through all four calls, a slot given back between the steps."""
    B, K, V, R = 6, 3, 1500, 11
    rng = np.random.default_rng(3)
    h = Head(512, V, 64, True, "bfloat16", seed=3)
    dev = lambda x: torch.as_tensor(np.ascontiguousarray(x)).cuda()  # noqa: E731
    history, want = sv.TokenHistory.empty(R, V, "cuda"), plain.History(R, V)
    slot = rng.permutation(R)[:B].astype(np.int32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    prompt = rng.integers(0, V, (B, 20)).astype(np.int32)
    sv.sv_history_add(history, dev(prompt), kind=sv.SV_HISTORY_PROMPT, slots=dev(slot), status=st)
    for b in range(B):
        want.add(slot[b], prompt[b], prompt=True)
    pen = [rng.uniform(lo, hi, B).astype(np.float32) for lo, hi in ((1, 1.5), (0, 0.4), (0, 0.4))]
    ws = torch.empty(max(16, sv.sv_head_w4_workspace_bytes(h.weight, B, K + 1)), dtype=torch.uint8,
                     device="cuda")
    for step in range(3):
        lengths = rng.integers(0, K + 1, B).astype(np.int32)
        drafts = rng.integers(0, V, (B, K)).astype(np.int32)
        allowed = rng.random((2, V)) < 0.7
        index = rng.integers(-1, 2, (B, K + 1)).astype(np.int32)
        rules = sv.LogitRules(history, dev(slot), *map(dev, pen), mask=dev(plain.pack(allowed)),
                              mask_index=dev(index))
        x, ln, dr = h.x(B, K + 1), dev(lengths), dev(drafts)
        zt, zd = torch.zeros(B, K + 1, V, device="cuda"), torch.randn(B, K, V, device="cuda")
        sv.sv_head_w4(h.weight, x, zt, ws, lengths=ln, extra=1, status=st)
        raw = zt.double().cpu().numpy()
        sv.sv_logits_process(zt, zt, rules, dr, ln, extra=1, status=st)
        tokens, accepted = sv.verify(zt, zd, dr, ln, torch.ones(B, device="cuda"), seed=step, status=st)
        sv.sv_history_add(history, tokens, lens=accepted, extra=1, slots=dev(slot), status=st)
        assert int(st) & ~(sv.SV_NOTE_CDF_FALLBACK | sv.SV_NOTE_ZERO_RESIDUAL) == 0
        got, tok, acc = zt.double().cpu().numpy(), tokens.cpu().numpy(), accepted.cpu().numpy()
        for b in range(B):
            s, n = slot[b], int(lengths[b]) + 1
            masks = [allowed[i] if i >= 0 else None for i in index[b]]
            out, bound = plain.process(raw[b], "float32", drafts[b], 0, n, want.prompt[s], want.counts[s],
                                       *(float(p[b]) for p in pen), {}, masks)
            plain.check(got[b], out, bound)
            want.add(s, tok[b, :acc[b] + 1])
        sv.sv_history_reset(history, slots=dev(slot[step:step + 1]), status=st)
        want.counts[slot[step]], want.prompt[slot[step]] = 0, False
        assert np.array_equal(history.output_counts.cpu().numpy(), want.counts)
        assert np.array_equal(history.output_bits.cpu().numpy(), plain.pack(want.counts > 0))
        assert np.array_equal(history.prompt_bits.cpu().numpy(), plain.pack(want.prompt))


@pytest.mark.parametrize("seed", range(60))
def test_heads_of_random_sizes(seed):
    rng = np.random.default_rng(2000 + seed)
    group = int(rng.choice([32, 64, 128]))
    H = group * int(np.exp(rng.uniform(0, np.log(8192 // group))))
    V = int(np.exp(rng.uniform(0, np.log(min(20000, 2e7 / H)))))
    P = int(rng.choice([1, 2, 3, 5, 9]))
    B = max(1, min(int(np.exp(rng.uniform(0, np.log(400)))), int(3e9 / (H * V)), 400) // P)
    h = Head(H, V, group, bool(rng.random() < 0.5), str(rng.choice(["float32", "bfloat16"])), seed)
    lengths = torch.from_numpy(rng.integers(-2, P + 3, B).astype(np.int32)).cuda() \
        if rng.random() < 0.5 else None
    h.check(h.x(B, P), str(rng.choice(["float32", "bfloat16"])), lengths, int(rng.integers(0, 2)))


def test_head_of_more_than_four_gigabytes_of_codes():
    V, H, group = 1 << 20, 8192, 32
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 256, (V, H // 2), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.rand(V, H // group, generator=g, device="cuda").bfloat16()
    zero = torch.randint(0, 16, (V, H // group), generator=g, device="cuda", dtype=torch.uint8)
    weight = sv.W4Weight(codes, scale, zero)
    # the first rows, those around 2 GB of codes, the last
    rows = torch.cat([torch.arange(a - 150, a + 150) for a in (150, V // 2, V - 150)]).cuda()
    sub = codes[rows].cpu().numpy()
    q = np.stack((sub & 15, sub >> 4), -1).reshape(len(rows), H)
    for M in (2, 20):
        x = torch.randn(M, 1, H, generator=g, device="cuda").bfloat16()
        out = torch.zeros(M, 1, V, device="cuda")
        need = sv.sv_head_w4_workspace_bytes(weight, M, 1)
        sv.sv_head_w4(weight, x, out, torch.empty(max(need, 16), dtype=torch.uint8, device="cuda"))
        want, bound = plain.head(x[:, 0].double().cpu().numpy(), q, scale[rows].double().cpu().numpy(),
                                 zero[rows].double().cpu().numpy(), group, "float32")
        plain.check(out[:, 0, rows].double().cpu().numpy(), want, bound)


def test_head_of_more_than_four_gigabytes_of_logits():
    V, M = 1 << 20, 2100
    h = Head(32, V, 32, False, "float32", seed=29)
    x = torch.randint(-3, 4, (M, 1, 32), dtype=torch.int8, device="cuda").bfloat16()
    out = torch.full((M, 1, V), 55.0, device="cuda")
    lengths = torch.ones(M, dtype=torch.int32, device="cuda")
    lengths[M - 2] = 0
    ws = torch.empty(sv.sv_head_w4_workspace_bytes(h.weight, M, 1), dtype=torch.uint8, device="cuda")
    sv.sv_head_w4(h.weight, x, out, ws, lengths=lengths)
    w = torch.from_numpy(h.codes.astype(np.float64) - 8).cuda() * h.scale.double().cuda()
    for m in (0, 1023, 1024, 2047, 2048, M - 1):
        want = (x[m].double() @ w.T)
        # integers of at most 32 * 3 * 8 are exact; the scale's product rounds once
        assert bool(((out[m].double() - want).abs() <= want.abs() * 2.0 ** -24).all())
    assert bool((out[M - 2] == 55).all())


@pytest.mark.parametrize("M", [3, 20, 140])
def test_head_of_weights_written_just_before(M):
    """Weights, scales and tokens that the stream writes right before each call."""
    heads = [Head(1024, 5000, 64, True, "bfloat16", seed=s) for s in (31, 32)]
    x = [h.x(M, 1) for h in heads]
    want = [h.want(t, "float32") for h, t in zip(heads, x)]
    w = [heads[0].weight.codes.clone(), heads[0].weight.scale.clone(), heads[0].weight.zero.clone()]
    weight, xs = sv.W4Weight(*w), x[0].clone()
    need = sv.sv_head_w4_workspace_bytes(weight, M, 1)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros(M, 1, 5000, device="cuda") for _ in range(6)]

    def write(i):
        for t, s in zip(w + [xs], (heads[i].weight.codes, heads[i].weight.scale, heads[i].weight.zero, x[i])):
            torch.add(s, 0, out=t) if t.dtype != torch.uint8 else torch.bitwise_or(s, 0, out=t)
    write(0)
    torch.cuda.synchronize()
    for n, out in enumerate(outs):
        write(n % 2)
        sv.sv_head_w4(weight, xs, out, ws)
    torch.cuda.synchronize()
    for n, out in enumerate(outs):
        plain.check(out.double().cpu().numpy(), *want[n % 2])


def test_chain_in_a_graph():
    """Head, rules, verification and history captured once and replayed: each
    replay goes on from the history that the one before left, as eager calls do."""
    B, K, V = 12, 4, 3001
    h = Head(512, V, 64, True, "bfloat16", seed=37)
    rng = np.random.default_rng(37)
    dev = lambda x: torch.as_tensor(np.ascontiguousarray(x)).cuda()  # noqa: E731
    slot, pen = dev(rng.permutation(B + 3)[:B].astype(np.int32)), [
        dev(rng.uniform(lo, hi, B).astype(np.float32)) for lo, hi in ((1, 1.5), (0, 0.4), (0, 0.4))]
    mask, index = dev(plain.pack(rng.random((3, V)) < 0.6)), dev(rng.integers(-1, 3, (B, K + 1)).astype(np.int32))
    x, ln = h.x(B, K + 1), dev(rng.integers(0, K + 1, B).astype(np.int32))
    dr, zd = dev(rng.integers(0, V, (B, K)).astype(np.int32)), torch.randn(B, K, V, device="cuda")
    temp = torch.ones(B, device="cuda")

    def side():
        """One copy of everything that a step writes, and the step."""
        history = sv.TokenHistory.empty(B + 3, V, "cuda")
        rules = sv.LogitRules(history, slot, *pen, mask=mask, mask_index=index)
        zt = torch.zeros(B, K + 1, V, device="cuda")
        tok = torch.zeros(B, K + 1, dtype=torch.int32, device="cuda")
        acc = torch.zeros(B, dtype=torch.int32, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        ws = torch.empty(max(16, sv.sv_head_w4_workspace_bytes(h.weight, B, K + 1)), dtype=torch.uint8, device="cuda")
        vws = torch.empty(sv.sv_verify_workspace_bytes(B, K, V, sv.SV_F32), dtype=torch.uint8, device="cuda")

        def step():
            sv.sv_head_w4(h.weight, x, zt, ws, lengths=ln, extra=1, status=st)
            sv.sv_logits_process(zt, zt, rules, dr, ln, extra=1, status=st)
            sv.sv_verify(zt, zd, dr, ln, temp, 5, tok, acc, vws, status=st)
            sv.sv_history_add(history, tok, lens=acc, extra=1, slots=slot, status=st)
        written = (zt, tok, acc, st, history.prompt_bits, history.output_bits, history.output_counts)
        return step, written
    eager, a = side()
    captured, b = side()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured()
    for _ in range(4):
        eager()
        graph.replay()
        torch.cuda.synchronize()
        for s, t in zip(a, b):
            assert torch.equal(s, t)
        assert int(a[3]) & ~(sv.SV_NOTE_CDF_FALLBACK | sv.SV_NOTE_ZERO_RESIDUAL) == 0
    assert int(a[6].sum()) >= 4 * B
