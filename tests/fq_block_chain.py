"""The transformer block that test_gpu_block.py runs: sites, buffers and the calls in order."""
import numpy as np
import torch

import blockref as ref
import w4a4_integer_gemm_amd as fq
from fqtest import dev


class Block:
    K, D, q_heads, kv_heads, F, eps = 512, 64, 4, 2, 640, 1e-6

    def __init__(self, M, f32, seed):
        rng = np.random.default_rng(seed)
        self.M, self.f32, self.rot_heads = M, f32, self.q_heads + self.kv_heads
        K, heads = self.K, self.q_heads + 2 * self.kv_heads
        w = lambda n, k: (rng.standard_normal((n, k)) * k ** -0.5).astype(np.float32)  # noqa: E731
        gain = lambda: rng.uniform(0.5, 1.5, K).astype(np.float32)  # noqa: E731
        self.g1_host, self.g2_host, self.g3_host = gain(), gain(), gain()
        self.g1, self.g2, self.g3 = dev(self.g1_host), dev(self.g2_host), dev(self.g3_host)
        self.qkv = fq.Fp8Site(w(heads * self.D, K))
        self.o = fq.Fp8Site(w(K, self.q_heads * self.D), bias=rng.standard_normal(K).astype(np.float32))
        self.up = fq.Fp8Site(w(2 * self.F, K))
        self.down = fq.Fp8Site(w(K, self.F))
        self.per = 5  # rows of one condition
        conds = -(-M // self.per)
        self.cond = dev(ref.bf16(rng, conds, 3 * K, scale=0.3))
        self.freq_host, _ = fq.fq_rope_freqs(self.D, 10000.0)
        self.freq = dev(self.freq_host.view(np.int64))
        empty = lambda *s: torch.empty(s, dtype=torch.int16, device="cuda")  # noqa: E731
        st = torch.float32 if f32 else torch.int16
        self.stream = torch.empty((M, K), dtype=st, device="cuda")
        self.stream1, self.stream2 = torch.empty_like(self.stream), torch.empty_like(self.stream)
        self.pos = torch.empty(M, dtype=torch.int32, device="cuda")
        self.codes1, self.scales1 = self.qkv.empty_codes(M)
        self.codes2, self.scales2 = self.up.empty_codes(M)
        self.qkv_out, self.heads = empty(heads, M, self.D), empty(heads, M, self.D)
        self.o_in, self.o_out = empty(M, self.q_heads * self.D), empty(M, K)
        self.up_out, self.mlp, self.down_out, self.h = empty(M, 2 * self.F), empty(M, self.F), empty(M, K), empty(M, K)
        self.o.workspace(M), self.down.workspace(M)
        self.new_inputs(rng)

    def new_inputs(self, rng):
        s = rng.standard_normal((self.M, self.K)).astype(np.float32) * 2
        self.stream.copy_(dev(s) if self.f32 else dev(ref.bf16(rng, self.M, self.K, scale=2)))
        self.pos.copy_(dev(rng.integers(0, 5000, self.M).astype(np.int32)))

    def run(self):
        M, K, D, e = self.M, self.K, self.D, self.eps
        fq.fq_block_norm(M, K, None, 0, None, 0.0, None, 0, 1.0, self.stream, K, None, 0, self.f32, self.g1, e, None,
                         None, 0, 1, None, 0, self.codes1, self.scales1)
        self.qkv.gemm(self.codes1, self.scales1, M, head_dim=D, y=self.qkv_out)
        self.heads.copy_(self.qkv_out)
        n = self.heads.shape[0]
        fq.fq_rope(self.heads, D, M * D, M, n, self.rot_heads, D, D, 0, self.freq, 1.0, self.pos, 0, 0, self.heads, D,
                   M * D)
        self.o_in.view(M, self.q_heads, D).copy_(self.heads[:self.q_heads].transpose(0, 1))
        self.o.linear(self.o_in, y=self.o_out)
        c = self.cond
        fq.fq_block_norm(M, K, self.o_out, K, self.g2, e, c[:, 2 * K:], 3 * K, 0.5, self.stream, K, self.stream1, K,
                         self.f32, None, e, c[:, :K], c[:, K:2 * K], 3 * K, self.per, None, 0, self.codes2, self.scales2)
        self.up.gemm(self.codes2, self.scales2, M, y=self.up_out)
        fq.fq_geglu(self.up_out, M, self.F, 2 * self.F, self.mlp, self.F)
        self.down.linear(self.mlp, y=self.down_out)
        self.stream2.copy_(self.stream1)
        fq.fq_block_norm(M, K, self.down_out, K, self.g3, e, None, 0, 1.0, self.stream2, K, self.stream2, K, self.f32,
                         self.g1, e, None, None, 0, 1, self.h, K)

    def outputs(self):
        return (self.codes1, self.scales1[:, :self.M], self.heads, self.o_out, self.stream1, self.codes2,
                self.scales2[:, :self.M], self.up_out, self.down_out, self.stream2, self.h)

    def poison(self):
        for t in self.outputs():
            t.fill_(77)
