"""One attention sublayer served with the library: a prompt, then decode and verify steps.

    python examples/attention_step.py [--steps]

A batch of sequences runs through the calls a serving program makes per step:

    qg_cache_pages     slots and block table of the step's new tokens
    qgemv              query / key / value projection, 2560 -> 10240 (48 + 16 + 16 heads of 128)
    qg_cache_append    norm, rotation, keys and values into the 4-bit cache, queries out
    qg_attention       the new tokens over the cache
    qgemv              output projection, 6144 -> 2560

The prompts go in whole, with qgemm for qgemv and qg_prompt_attention over the keys and values as the
cache has stored them, or (--steps) two tokens of each at a time through the same calls as the decode
step; weights and inputs are random.  The decode step is captured once as a CUDA graph and replayed:
nothing in it reads back to the host, and the lengths live on the device.
"""
from __future__ import annotations

import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import block_quantized_token_format_gb300 as qg  # noqa: E402

D_MODEL, HEADS, KV, DIM, PAGE = 2560, 48, 16, 128, 64
QKV = (HEADS + 2 * KV) * DIM


class AttentionLayer:
    """Weights, rotation table and workspace of one layer, on the current device."""

    def __init__(self, seed: int, n_pages: int, n_pos: int = 4096):
        g = np.random.default_rng(seed)

        def packed(n_out, n_in):
            return torch.from_numpy(qg.qg_pack("q8_0", g.standard_normal((n_out, n_in), dtype=np.float32) * 0.02)).cuda()

        self.w_qkv, self.w_out = packed(QKV, D_MODEL), packed(D_MODEL, HEADS * DIM)
        self.q_weight, self.k_weight = [torch.from_numpy(1 + 0.1 * g.standard_normal(DIM).astype(np.float32)).cuda() for _ in range(2)]
        angle = np.outer(np.arange(n_pos), 1e6 ** (-np.arange(0, DIM, 2) / DIM))
        self.cos_sin = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).cuda()
        pool = torch.empty(qg.qg_cache_bytes(n_pages, PAGE, KV, DIM), dtype=torch.uint8, device="cuda")
        self.cache = qg.qg_cache(pool, n_pages, PAGE, KV, DIM)
        self.workspace = torch.zeros(qg.qg_attention_workspace_bytes(HEADS, KV, DIM), dtype=torch.uint8, device="cuda")

    def __call__(self, x, step):
        """x: fp32 ``[n_tok, 2560]`` (at most 4 rows) -> the sublayer's output, same shape."""
        n = x.shape[0]
        qkv = torch.empty(n, HEADS + 2 * KV, DIM, device="cuda")
        qg.qgemv("q8_0", self.w_qkv, QKV, D_MODEL, x, qkv, n)
        q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], qkv[:, HEADS + KV:]
        qg.qg_cache_append(self.cache, k, v, step.slots, q=q, q_out=q, positions=step.positions, cos_sin=self.cos_sin,
                           q_weight=self.q_weight, k_weight=self.k_weight)
        out = torch.empty(n, HEADS, DIM, device="cuda")
        qg.qg_attention(self.cache, q, step.table, step.seq_len, step.cu_new, out, self.workspace, DIM ** -0.5, max_new=step.max_new)
        y = torch.empty_like(x)
        qg.qgemv("q8_0", self.w_out, D_MODEL, HEADS * DIM, out, y, n)
        return y


    def prompt(self, x, step):
        """The same for whole prompts, packed: x fp32 ``[n_tok, 2560]``; the cache holds nothing of them before."""
        n = x.shape[0]
        work = max(qg.qgemm_workspace_bytes("q8_0", "f32", QKV, D_MODEL, n), qg.qgemm_workspace_bytes("q8_0", "f32", D_MODEL, HEADS * DIM, n),
                   qg.qg_prompt_attention_workspace_bytes("f32", n, HEADS, KV, DIM))
        work = torch.empty(work, dtype=torch.uint8, device="cuda")               # one after the other: one workspace
        qkv = torch.empty(n, HEADS + 2 * KV, DIM, device="cuda")
        qg.qgemm("q8_0", self.w_qkv, QKV, D_MODEL, x, qkv.view(n, QKV), work)
        q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], qkv[:, HEADS + KV:]
        k_back, v_back = [torch.empty(n, KV, DIM, device="cuda") for _ in range(2)]
        qg.qg_cache_append(self.cache, k, v, step.slots, q=q, q_out=q, positions=step.positions, cos_sin=self.cos_sin,
                           q_weight=self.q_weight, k_weight=self.k_weight, k_back=k_back, v_back=v_back)
        out = torch.empty(n, HEADS, DIM, device="cuda")
        qg.qg_prompt_attention(q, k_back, v_back, step.cu_new, out, work, DIM ** -0.5, longest=step.max_new)
        y = torch.empty_like(x)
        qg.qgemm("q8_0", self.w_out, D_MODEL, HEADS * DIM, out.view(n, HEADS * DIM), y, work)
        return y


class Step:
    """Device state of a batch: lengths, block table, free pages, and the current step's tokens."""

    def __init__(self, n_req: int, n_pages: int, width: int, fresh):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.held, self.fresh = torch.zeros(n_req, **i32), torch.tensor(fresh, **i32)
        self.table = torch.full((n_req, width), -1, **i32)
        self.free, self.begin = torch.randperm(n_pages, device="cuda").int(), torch.zeros(1, **i32)
        self.seq_len, self.cu_new = torch.zeros(n_req, **i32), torch.zeros(n_req + 1, **i32)
        self.set_fresh(fresh)

    def set_fresh(self, fresh):
        self.fresh.copy_(torch.tensor(fresh, dtype=torch.int32))
        self.max_new, n = max(fresh), sum(fresh)
        self.slots = torch.zeros(n, dtype=torch.int64, device="cuda")
        self.positions = torch.zeros(n, dtype=torch.int32, device="cuda")

    def begin_step(self):
        qg.qg_cache_pages(self.held, self.fresh, self.free, self.table, self.seq_len, self.cu_new, self.slots, self.positions,
                          PAGE, free_begin=self.begin, free_end=self.begin)

    def end_step(self):
        self.held.copy_(self.seq_len)


def main(prompt: int = 40, decode: int = 8, whole: bool = True) -> dict:
    torch.manual_seed(0)
    n_pages = 64
    layer, step = AttentionLayer(1, n_pages), Step(2, n_pages, 16, [prompt, prompt])
    tokens = torch.randn(2, prompt, D_MODEL, device="cuda")
    if whole:
        # Prompt: two sequences in one pass.
        step.begin_step()
        prompts = layer.prompt(tokens.view(2 * prompt, D_MODEL), step).view(2, prompt, D_MODEL)
        step.end_step()
    else:
        # Prompt: two sequences, two tokens each per step.
        prompts = torch.empty_like(tokens)
        for at in range(0, prompt, 2):
            now = tokens[:, at:at + 2].contiguous()
            step.set_fresh([now.shape[1]] * 2)
            step.begin_step()
            prompts[:, at:at + 2] = layer(now.view(-1, D_MODEL), step).view_as(now)
            step.end_step()
    # Decode: one token each, as one graph.
    step.set_fresh([1, 1])
    x = torch.randn(2, D_MODEL, device="cuda")

    def decode_step():
        step.begin_step()
        y = layer(x, step)
        step.end_step()
        return y

    decode_step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = decode_step()
    for _ in range(decode - 1):
        graph.replay()
    # Verify: four drafted tokens of the first sequence.
    step.set_fresh([4, 0])
    step.begin_step()
    z = layer(torch.randn(4, D_MODEL, device="cuda"), step)
    step.end_step()
    torch.cuda.synchronize()
    assert qg.qg_device_status() == 0
    return {"lengths": step.seq_len.tolist(), "pages": int(step.begin), "prompt": prompts, "decode": y, "verify": z}


if __name__ == "__main__":
    r = main(whole="--steps" not in sys.argv[1:])
    print("lengths", r["lengths"], "pages dealt", r["pages"], "output rms", float(r["verify"].square().mean().sqrt()))
