"""Serving a stack that mixes gated-delta-rule layers with softmax attention.

Three gated-delta-rule mixers for each attention mixer, as such models have
them.  The prompts of a batch are packed and run through gdn_chunk_fwd, whose
final states gdn_decode_step then advances token by token; the attention
mixers keep an 8-bit key/value cache instead (gdn_kv_append, gdn_kv_attn).  The
decode step is captured once as a CUDA graph: its lengths and page table are
device data, so replays follow the growing sequences.

The projections are plain bf16 matrix products with random weights; only the
mixers are the point.  Run it on a GPU:

    python examples/hybrid_layers.py
"""
from __future__ import annotations

import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gated_deltanet_linear_fwd_gb300 as gdn  # noqa: E402

D = 128      # elements of a head
PAGE = 64    # tokens of a cache page


def _weight(gen, rows, cols):
    return (torch.randn(rows, cols, device="cuda", generator=gen) / cols ** 0.5).bfloat16()


class DeltaMixer:
    """o = W_o . gated_delta_rule(q, k, v, g, beta), all from projections of x."""

    def __init__(self, gen, width, h_qk, h_v):
        self.h_qk, self.h_v = h_qk, h_v
        self.w_in = _weight(gen, (2 * h_qk + h_v) * D, width)
        self.w_gate = _weight(gen, 2 * h_v, width)
        self.w_out = _weight(gen, width, h_v * D)
        self.state = None

    def _project(self, x):
        qkv = (x @ self.w_in.T).view(-1, 2 * self.h_qk + self.h_v, D)
        q, k, v = qkv.split([self.h_qk, self.h_qk, self.h_v], dim=1)
        gate = (x @ self.w_gate.T).float()
        g = F.logsigmoid(gate[:, :self.h_v] + 3.0)
        beta = torch.sigmoid(gate[:, self.h_v:])
        unit = lambda t: F.normalize(t.float(), dim=-1).bfloat16()  # noqa: E731
        return unit(q), unit(k), v.contiguous(), g.contiguous(), beta.contiguous()

    def prefill(self, x, cu_seqlens):
        # a captured step goes on reading the first states' memory
        o, self.state = gdn.gdn_chunk_fwd(*self._project(x), None, cu_seqlens, final_state=self.state)
        return o.flatten(1) @ self.w_out.T

    def step(self, x):
        return gdn.gdn_decode_step(*self._project(x), self.state).flatten(1) @ self.w_out.T


class AttentionMixer:
    """o = W_o . softmax attention over an 8-bit cache."""

    def __init__(self, gen, width, h_q, h_kv, n_pages):
        self.h_q, self.h_kv = h_q, h_kv
        self.w_in = _weight(gen, (h_q + 2 * h_kv) * D, width)
        self.w_out = _weight(gen, width, h_q * D)
        self.cache = gdn.KVCache.empty(n_pages, h_kv)

    def __call__(self, x, kv_lens, page_table, cu_seqlens=None, *, plan=None, workspace=None):
        # the heads of one fused projection are used in place, by their strides
        qkv = (x @ self.w_in.T).view(-1, self.h_q + 2 * self.h_kv, D)
        q, k, v = qkv.split([self.h_q, self.h_kv, self.h_kv], dim=1)
        gdn.gdn_kv_append(self.cache, k, v, kv_lens, page_table, cu_seqlens)
        o, _ = gdn.gdn_kv_attn(q, self.cache, kv_lens, page_table, cu_seqlens, plan=plan, workspace=workspace,
                               return_lse=False)
        return o.flatten(1) @ self.w_out.T


class HybridStack:
    """Every fourth mixer is attention.  One page table serves all of them."""

    def __init__(self, n_layers=8, width=512, h_qk=2, h_v=8, h_q=8, h_kv=2, max_tokens=4096, batch=4, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        pages = -(-max_tokens // PAGE)
        self.batch, self.pages = batch, pages
        self.h_q, self.h_kv = h_q, h_kv
        self.layers = [AttentionMixer(gen, width, h_q, h_kv, batch * pages) if i % 4 == 3
                       else DeltaMixer(gen, width, h_qk, h_v) for i in range(n_layers)]
        # any assignment will do; a serving program hands pages out as sequences grow
        self.page_table = torch.randperm(batch * pages, device="cuda", generator=gen).to(torch.int32).view(batch, pages)
        self.kv_lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.graph = None

    def prefill(self, x, lens):
        """x [sum(lens), width]: the prompts, packed.  Returns the stack's output for every token."""
        cu = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()
        self.kv_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        for layer in self.layers:
            y = layer.prefill(x, cu) if isinstance(layer, DeltaMixer) else layer(x, self.kv_lens, self.page_table, cu)
            x = x + y
        return x

    def _step(self, x, plan, workspace):
        for layer in self.layers:
            y = layer.step(x) if isinstance(layer, DeltaMixer) else layer(x, self.kv_lens, self.page_table, plan=plan,
                                                                          workspace=workspace)
            x = x + y
        return x

    def step(self, x):
        """x [batch, width]: one more token of each sequence."""
        self.kv_lens += 1
        if self.graph is None:
            plan = gdn.gdn_kv_attn_plan(T=self.batch, n_seqs=self.batch, h_q=self.h_q, h_kv=self.h_kv, max_q_len=1,
                                        max_pages=self.pages)
            workspace = torch.empty(max(256, plan.workspace_bytes), dtype=torch.uint8, device="cuda")
            self.x = x.clone()
            states = [layer.state.clone() for layer in self.layers if isinstance(layer, DeltaMixer)]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):  # warm-up, and undo what it did to the states (the cache's tokens are rewritten)
                self._step(self.x, plan, workspace)
                for layer, s in zip((m for m in self.layers if isinstance(m, DeltaMixer)), states):
                    layer.state.copy_(s)
            torch.cuda.current_stream().wait_stream(side)
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.y = self._step(self.x, plan, workspace)
            self.keep = (plan, workspace)
        self.x.copy_(x)
        self.graph.replay()
        return self.y


def main():
    lens, steps, width = [700, 64, 1, 1290], 20, 512
    gen = torch.Generator("cuda").manual_seed(1)
    stack = HybridStack(width=width, batch=len(lens))
    x = torch.randn(sum(lens), width, device="cuda", generator=gen).bfloat16()
    y = stack.prefill(x, lens)
    for _ in range(steps):
        y = stack.step(torch.randn(len(lens), width, device="cuda", generator=gen).bfloat16())
    torch.cuda.synchronize()
    for layer in stack.layers:
        if isinstance(layer, AttentionMixer):
            code, detail = gdn.gdn_get_device_status(layer.cache.status)
            assert code == 0, gdn.describe_device_status(code, detail)
    print(f"prompts of {lens} tokens, then {steps} steps: lengths {stack.kv_lens.tolist()}, output {tuple(y.shape)}")


if __name__ == "__main__":
    main()
