"""A decode step with its attention and its choice of the next token, as a loop over
several sequences runs it: norm_quant and an 8-bit projection for queries, keys
and values, kv_append, kv_attend, a projection back, the head, logits_process,
sample and the embedding of the drawn tokens.

Each operator is compared with the float64 oracle on what the one before it left
on the GPU, with the bounds of its own tests; the cache of each step is what the
steps before wrote."""
import numpy as np
import pytest

import bit_affine_quantized_gb300 as bq
from kv_cases import BF16, F32, f64, i32
from oracle import batch_oracle as BO
from oracle import head_oracle as HO
from oracle import kv_oracle as KO
from synth.device import DeviceHead
from test_gpu_kv_attend import check as check_attend
from test_gpu_kv_cache import TURN, near
from test_gpu_norm_quant import REL, dev16, host16, rows
from test_gpu_qdense import bound, codes
from test_gpu_sample import check as check_sample

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

H, V = 512, 2064  # V: rows of the tied 4-bit embedding, a multiple of 16
PAGE, D, HQ, HKV, ROT = 16, 64, 6, 2, 32


class Loop:
    def __init__(self, moe, T, bits8, seed=0):
        self.moe, self.T, self.bits8 = moe, T, bits8
        g = np.random.default_rng(seed + T)
        self.rng = g
        widths = {"qkv": ((HQ + 2 * HKV) * D, H), "o": (H, HQ * D), "head": (V, H)}
        self.w, self.ws, self.wd, work = {}, {}, {}, 0
        for i, (name, (n, k)) in enumerate(widths.items()):
            self.w[name] = codes(seed + 10 * T + i, n, k)
            self.ws[name] = (g.uniform(0.5, 1.0, n) * 3 / np.sqrt(k)).astype(np.float32) / 127
            if name == "head":
                self.ws[name] *= 127 / 40
            self.wd[name] = bq.make_qdense_weights(n, k, torch.from_numpy(self.w[name]).cuda(),
                                                   torch.from_numpy(self.ws[name]).cuda())
            work = max(work, moe.qdense_workspace_bytes(self.wd[name], T))
        self.work = torch.empty(work, dtype=torch.uint8, device="cuda")
        self.emb = DeviceHead(7, V, H)
        self.hw = bq.make_head_weights(V, H, *self.emb.addresses())
        # the cache: prompts of different lengths, the pages of sequences interleaved
        self.lengths0 = g.integers(0, 60, T)
        self.lengths0[0] = 0
        per = 5
        self.table = g.permutation(T * per + 3)[:T * per].reshape(T, per).astype(np.int32)
        shape = (T * per + 3, HKV, PAGE, D)
        kind = torch.int8 if bits8 else torch.bfloat16
        self.k, self.v = torch.zeros(shape, dtype=kind, device="cuda"), torch.zeros(shape, dtype=kind, device="cuda")
        self.ks = torch.zeros(shape[:3], device="cuda") if bits8 else None
        self.vs = torch.zeros(shape[:3], device="cuda") if bits8 else None
        self.cache = bq.make_kv_cache(self.k, self.v, i32(self.table), self.ks, self.vs)
        self.freq_host = (10000.0 ** (-np.arange(0, ROT, 2) / ROT)).astype(np.float32)
        self.freq = torch.from_numpy(self.freq_host).cuda()
        self.ws_attend = torch.empty(moe.kv_attend_workspace_bytes(self.cache, HQ), dtype=torch.uint8, device="cuda")
        seq = np.repeat(np.arange(T), self.lengths0)
        pos = np.concatenate([np.arange(n) for n in self.lengths0]).astype(int)
        prompt = torch.from_numpy(g.standard_normal((max(len(seq), 1), 2, HKV, D))).to(torch.bfloat16).cuda()
        if len(seq):
            moe.kv_append(prompt[:, 0].contiguous(), prompt[:, 1].contiguous(), i32(pos), self.cache, seqs=i32(seq),
                          inv_freq=self.freq)
        # what a step reads and writes
        e = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")
        self.hidden, self.y = dev16(rows(T + 1, T, H)), dev16(rows(T + 2, T, H))
        self.pos, self.len = i32(self.lengths0), i32(self.lengths0 + 1)
        self.q8, self.s8 = e(T, H, dtype=torch.int8), e(T)
        self.qkv, self.q = e(T, (HQ + 2 * HKV) * D, dtype=torch.bfloat16), e(T, HQ, D, dtype=torch.bfloat16)
        self.out, self.lse = e(T, HQ * D, dtype=torch.bfloat16), e(T, HQ)
        self.o8, self.os = e(T, HQ * D, dtype=torch.int8), e(T)
        self.h8, self.hs = e(T, H, dtype=torch.int8), e(T)
        self.logits, self.tokens, self.logp = e(T, V), e(T, dtype=torch.int32), e(T)
        self.temp = g.uniform(0.5, 1.5, T).astype(np.float32)
        self.top_k, self.top_p = g.integers(0, 40, T).astype(np.int32), g.uniform(0.5, 1.2, T).astype(np.float32)
        self.u = torch.zeros(T, device="cuda")
        self.rules = bq.make_sample_rules(self.u, torch.from_numpy(self.temp).cuda(), torch.from_numpy(self.top_k).cuda(),
                                          torch.from_numpy(self.top_p).cuda())
        self.hist = torch.zeros((T, 8), dtype=torch.int32, device="cuda")
        self.logit_rules = bq.make_logit_rules(history=self.hist, history_len=torch.full((T,), 8, dtype=torch.int32, device="cuda"),
                                               repetition=torch.full((T,), 1.5, device="cuda"))
        self.next = torch.empty((T, H), dtype=torch.int16, device="cuda")

    def step(self, stream=None):
        m, T, kw = self.moe, self.T, dict(stream=stream)
        m.norm_quant(self.hidden, T, self.q8, self.s8, y=self.y, hidden_out=self.hidden, **kw)
        m.qdense_forward(self.q8, self.s8, T, self.wd["qkv"], self.work, y=self.qkv, **kw)
        q, k, v = self.qkv.split((HQ * D, HKV * D, HKV * D), 1)
        m.kv_append(k, v, self.pos, self.cache, q=q, q_out=self.q, inv_freq=self.freq, **kw)
        m.kv_attend(self.q, self.len, self.cache, self.out, self.ws_attend, scale=D ** -0.5, lse=self.lse, **kw)
        m.norm_quant(self.out, T, self.o8, self.os, **kw)
        m.qdense_forward(self.o8, self.os, T, self.wd["o"], self.work, y=self.y, **kw)
        m.norm_quant(self.hidden, T, self.h8, self.hs, y=self.y, hidden_out=self.hidden, **kw)
        m.qdense_forward(self.h8, self.hs, T, self.wd["head"], self.work, y32=self.logits, softcap=30.0, **kw)
        m.logits_process(self.logits, T, V, self.logit_rules, out=self.logits, **kw)
        m.sample(self.logits, T, V, self.rules, self.tokens, logprobs=self.logp, **kw)
        m.embed(self.tokens, T, self.hw, self.next, **kw)

    def check(self, pages_before):
        T = self.T
        at = self.pos.cpu().numpy()
        qkv = f64(self.qkv)
        z = BO.qdense(self.q8.cpu().numpy(), self.s8.cpu().numpy(), self.w["qkv"], self.ws["qkv"])
        assert np.all(np.abs(qkv - z) <= bound(self.q8.cpu().numpy(), self.w["qkv"], self.s8.cpu().numpy(), self.ws["qkv"])
                      + BF16 * np.abs(z) * 1.01)
        q, k, v = (qkv[:, a:b].reshape(T, -1, D) for a, b in
                   ((0, HQ * D), (HQ * D, (HQ + HKV) * D), ((HQ + HKV) * D, (HQ + 2 * HKV) * D)))
        assert near(f64(self.q), KO.rotate(q, at, self.freq_host), q, ROT)
        # the new rows, and nothing else, in the pages
        page, row = self.table[np.arange(T), at // PAGE], at % PAGE
        pk, pv = f64(self.k), f64(self.v)
        for before, now in zip(pages_before, (pk, pv)):
            was = before.copy()
            was[page, :, row] = now[page, :, row]
            assert np.array_equal(was, now)
        turned = KO.rotate(k, at, self.freq_host)
        if self.bits8:
            ks = f64(self.ks)
            most = 2 * np.abs(k).max(-1)[..., None]
            s = ks[page, :, row][..., None]
            assert np.all(np.abs(pk[page, :, row] * s - turned) <= s * (0.5 + 600 * F32) + 2 * TURN * most)
            assert np.array_equal(pv[page, :, row], KO.quantise(v)[0])
        else:
            assert near(pk[page, :, row], turned, k, ROT) and np.array_equal(pv[page, :, row], v)

        class Host:  # the cache as it stands on the GPU
            heads, bits8 = HKV, self.bits8

            @staticmethod
            def rows(seq, pos):
                sk, sv = (f64(self.ks), f64(self.vs)) if self.bits8 else (None, None)
                return (KO.rows(pk, sk, self.table, PAGE, seq, pos), KO.rows(pv, sv, self.table, PAGE, seq, pos))
        check_attend(Host, f64(self.q), at + 1, D ** -0.5, 0.0, 0, self.out, self.lse)
        want = BO.norm_quant(host16(self.out.view(torch.int16)))
        assert np.array_equal(self.o8.cpu().numpy(), want["q"])
        assert np.all(np.abs(f64(self.os) - want["scales"]) <= REL * want["scales"])
        lg, tk = self.logits.cpu().numpy(), self.tokens.cpu().numpy()
        check_sample(lg, tk, self.logp.cpu().numpy().astype(float), self.u.cpu().numpy(), self.temp, self.top_k, self.top_p)
        assert np.array_equal(host16(self.next), HO.embed(np.arange(T), self.emb.host_rows(tk)))
        return tk

    def advance(self, tk, step):
        self.pos += 1
        self.len += 1
        self.hist[:, step] = torch.from_numpy(tk).cuda()
        self.y.copy_(self.next)

    def pages(self):
        return f64(self.k), f64(self.v)

    def draw(self):
        self.u.copy_(torch.from_numpy(self.rng.random(self.T).astype(np.float32)))


@pytest.fixture(scope="module")
def moe():
    bq.build_library()
    m = bq.Moe()
    yield m
    m.close()


@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("T", [1, 5, 24])
def test_decode_loop(moe, T, bits8):
    loop = Loop(moe, T, bits8)
    for step in range(3):
        loop.draw()
        before = loop.pages()
        loop.step()
        torch.cuda.synchronize()
        assert moe.get_error() == bq.MOE_OK
        loop.advance(loop.check(before), step)


@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("T", [3, 24])
def test_decode_step_captured_by_a_new_handle(T, bits8):
    """The first calls that a handle sees of these operators are captured; the replays follow the buffers."""
    bq.build_library()
    moe = bq.Moe()
    loop = Loop(moe, T, bits8, seed=50)
    start = [t.clone() for t in (loop.hidden, loop.y)]
    pages = [t.clone() for t in (loop.k, loop.v)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            loop.step(stream=st)
        for a, b in zip((loop.hidden, loop.y, loop.k, loop.v), start + pages):
            a.copy_(b)
        for step in range(3):
            loop.draw()
            st.synchronize()
            before = loop.pages()
            g.replay()
            st.synchronize()
            assert moe.get_error() == bq.MOE_OK
            loop.advance(loop.check(before), step)
    moe.close()


@pytest.mark.parametrize("pdl", ["0"])
def test_decode_loop_without_early_launches(monkeypatch, pdl):
    monkeypatch.setenv("MOE_PDL", pdl)
    moe = bq.Moe()
    loop = Loop(moe, 5, True, seed=90)
    for step in range(2):
        loop.draw()
        before = loop.pages()
        loop.step()
        torch.cuda.synchronize()
        assert moe.get_error() == bq.MOE_OK
        loop.advance(loop.check(before), step)
    moe.close()


def test_a_prompt_in_chunks_and_a_ring_of_pages(moe):
    """A sliding window over a ring: the table names the same pages again, the oldest rows give way.  Chunks of a
    prompt are appended, the last token of each attends over the window."""
    W, n = 40, 4  # the window, the ring's pages: 64 rows hold a window and a chunk of 16 more
    g = np.random.default_rng(1)
    total = 200
    per = (total + PAGE - 1) // PAGE
    ring = g.permutation(9)[:n].astype(np.int32)
    table = ring[np.arange(per) % n][None]
    k = torch.zeros((9, HKV, PAGE, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    c = bq.make_kv_cache(k, v, i32(table))
    K, Vv = (torch.from_numpy(g.standard_normal((total, HKV, D))).to(torch.bfloat16) for _ in range(2))
    ws = torch.empty(moe.kv_attend_workspace_bytes(c, HQ), dtype=torch.uint8, device="cuda")

    class Host:
        heads, bits8 = HKV, False

        @staticmethod
        def rows(seq, pos):
            return K.double().numpy()[pos], Vv.double().numpy()[pos]
    for a in range(0, total, 16):
        b = min(total, a + 16)
        moe.kv_append(K[a:b].cuda(), Vv[a:b].cuda(), i32(np.arange(a, b)), c, seqs=i32(np.zeros(b - a)))
        q = torch.from_numpy(g.standard_normal((1, HQ, D))).to(torch.bfloat16)
        out, lse = torch.empty((1, HQ, D), dtype=torch.bfloat16, device="cuda"), torch.empty((1, HQ), device="cuda")
        moe.kv_attend(q.cuda(), i32([b]), c, out, ws, scale=0.125, window=W, lse=lse)
        assert moe.get_error() == bq.MOE_OK
        check_attend(Host, q.double().numpy(), [b], 0.125, 0.0, W, out, lse)
