"""The batched way from the residual stream to the next token on a GB300, as a
decode loop over many sequences uses it: norm_quant (the last layer's output
added, the final norm, 8-bit rows), qdense_forward (the 8-bit head with its
softcap), logits_process (penalties, biases, a grammar) and the embedding of
the chosen tokens, step after step.

Each operator is compared with the float64 oracle on what the one before it
left on the GPU, with the bounds of its own tests."""
import os

import numpy as np
import pytest

import bit_affine_quantized_gb300 as bq
from oracle import batch_oracle as BO
from oracle import head_oracle as HO
from synth.device import DeviceHead
from test_gpu_logits import check as check_logits
from test_gpu_logits import cuda, pack
from test_gpu_norm_quant import check as check_norm
from test_gpu_norm_quant import dev16, host16, rows
from test_gpu_qdense import F32, bound, codes

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

H, V = 768, 4112  # V: rows of the tied 4-bit embedding, a multiple of 16


class Loop:
    """One step of a decode loop over T sequences, all in one stream."""

    def __init__(self, moe, T, steps):
        self.moe, self.T = moe, T
        rng = np.random.default_rng(T)
        self.w, self.ws = codes(T, V, H), rng.uniform(0.002, 0.004, V).astype(np.float32)
        self.gamma = BO.to_bf16(rng.uniform(0.5, 1.5, H))
        self.wd = bq.make_qdense_weights(V, H, cuda(self.w), cuda(self.ws))
        self.work = torch.empty(moe.qdense_workspace_bytes(self.wd, T), dtype=torch.uint8, device="cuda")
        self.emb = DeviceHead(5, V, H)
        q, s, b = self.emb.addresses()
        self.hw = bq.make_head_weights(V, H, q, s, b)
        self.hidden, self.y = dev16(rows(T + 1, T, H)), dev16(rows(T + 2, T, H))
        self.q = torch.empty((T, H), dtype=torch.int8, device="cuda")
        self.scales = torch.empty(T, device="cuda")
        self.logits = torch.empty((T, V), device="cuda")
        self.out, self.tokens = torch.empty_like(self.logits), torch.empty(T, dtype=torch.int32, device="cuda")
        self.next = torch.empty((T, H), dtype=torch.int16, device="cuda")
        prompt = 7
        self.hist = torch.zeros((T, prompt + steps), dtype=torch.int32, device="cuda")
        self.hist[:, :prompt] = cuda(rng.integers(0, V, (T, prompt)).astype(np.int32))
        self.len = torch.full((T,), prompt, dtype=torch.int32, device="cuda")
        self.plen = self.len.clone()
        pen = [np.full(T, v, np.float32) for v in (1.25, 0.5, 0.25)]
        self.rep, self.pres, self.freq = (cuda(v) for v in pen)
        self.mask = rng.random((T, V)) < 0.5
        if T > 2:
            self.mask[2] = False  # a dead end
        self.bias_ids = cuda(rng.integers(0, V, (T, 3)).astype(np.int32))
        self.bias_values = cuda(rng.standard_normal((T, 3)).astype(np.float32))
        self.rules = bq.make_logit_rules(
            history=self.hist, history_len=self.len, prompt_len=self.plen, repetition=self.rep, presence=self.pres,
            frequency=self.freq, bias_ids=self.bias_ids, bias_values=self.bias_values,
            bias_len=torch.full((T,), 3, dtype=torch.int32, device="cuda"), mask=cuda(pack(self.mask)))

    def step(self, stream=None):
        m, T = self.moe, self.T
        m.norm_quant(self.hidden, T, self.q, self.scales, y=self.y, norm=cuda_gamma(self), hidden_out=self.hidden,
                     stream=stream)
        m.qdense_forward(self.q, self.scales, T, self.wd, self.work, y32=self.logits, softcap=30.0, stream=stream)
        m.logits_process(self.logits, T, V, self.rules, out=self.out, tokens=self.tokens, stream=stream)
        m.embed(self.tokens, T, self.hw, self.next, stream=stream)

    def check(self, before):
        T = self.T
        want = BO.norm_quant(before, host16(self.y), self.gamma)
        q, scales = self.q.cpu().numpy(), self.scales.cpu().numpy()
        check_norm({"s": host16(self.hidden), "q": q, "scales": scales.astype(np.float64), "x": None}, want)
        lg = self.logits.cpu().numpy()
        z = BO.qdense(q, scales, self.w, self.ws, 30.0)
        assert np.all(np.abs(lg - z) <= bound(q, self.w, scales, self.ws) + 12 * F32 * np.abs(z))
        hist, n, p = self.hist.cpu().numpy(), self.len.cpu().numpy(), self.plen.cpu().numpy()
        ids, vals = self.bias_ids.cpu().numpy(), self.bias_values.cpu().numpy().astype(float)
        rules = [dict(history=hist[t, :n[t]].tolist(), prompt=int(p[t]), repetition=1.25, presence=0.5, frequency=0.25,
                      bias=list(zip(ids[t].tolist(), vals[t].tolist()))) for t in range(T)]
        out, tk = self.out.cpu().numpy(), self.tokens.cpu().numpy()
        check_logits(lg, out, tk, rules, self.mask)
        fine = tk >= 0
        assert fine.sum() == T - (1 if T > 2 else 0)
        emb = host16(self.next)
        assert np.array_equal(emb[fine], HO.embed(np.arange(fine.sum()), self.emb.host_rows(tk[fine])))
        assert not emb[~fine].any()  # no token: a zero row
        return tk

    def advance(self, tk):
        """The tokens to the histories, their embeddings to the residual stream."""
        at = self.len.cpu().numpy()
        for t in np.flatnonzero(tk >= 0):
            self.hist[t, int(at[t])] = int(tk[t])
            self.len[t] += 1
        self.y.copy_(self.next)


def cuda_gamma(loop):
    if not hasattr(loop, "_gamma"):
        loop._gamma = dev16(loop.gamma[None])[0].contiguous()
    return loop._gamma


def _errors(moe, T):
    # a dead end has no token, and its embedding is recorded as a bad id
    assert moe.get_error() == (bq.MOE_ERR_BAD_EXPERT_ID if T > 2 else bq.MOE_OK)


@pytest.mark.parametrize("pdl", ["1", "0"])
@pytest.mark.parametrize("T", [1, 6, 24, 130])
def test_decode_loop(T, pdl):
    bq.build_library()
    old = os.environ.get("MOE_PDL")
    os.environ["MOE_PDL"] = pdl
    try:
        moe = bq.Moe()
    finally:
        if old is None:
            del os.environ["MOE_PDL"]
        else:
            os.environ["MOE_PDL"] = old
    loop = Loop(moe, T, 3)
    for _ in range(3):
        before = host16(loop.hidden)
        loop.step()
        torch.cuda.synchronize()
        _errors(moe, T)
        loop.advance(loop.check(before))
    moe.close()


@pytest.mark.parametrize("T", [3, 24])
def test_decode_step_captured_by_a_new_handle(T):
    """The first calls that a handle sees are captured; the replays follow what
    stands in the buffers."""
    bq.build_library()
    moe = bq.Moe()
    loop = Loop(moe, T, 2)
    cuda_gamma(loop)
    start = loop.hidden.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            loop.step(stream=st)
        loop.hidden.copy_(start)
        for _ in range(2):
            st.synchronize()
            before = host16(loop.hidden)
            g.replay()
            st.synchronize()
            _errors(moe, T)
            loop.advance(loop.check(before))
    moe.close()
