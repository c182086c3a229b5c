"""Verify steps of a speculative decoder over a paged cache, the library's calls
as they follow one another: a plan, then in every layer the append, the
attention of the drafted trees and the routed block.

    python -m mxfp4_mixture_experts_route_gb300.verify_step [--steps N] [--layers L] [--e4m3] [--projections]

With --projections a layer begins at its input rows: the fused query, key and value
projection with MXFP4 weights, the heads' norms and rotation with the append, the
attention, and the output projection (its rows quantised too) in front of the block.

The step is captured in one CUDA graph; lengths, trees, free pages and inputs
change between replays without a new capture, because the calls read them on
the device.  After a step a path of each tree is accepted: its K and V rows move
to the request's next slots (an append whose slot map names only them), and
pages past them go back to the free list.  There is no model around it: the
layers' q, k and v (or input rows) are seeded normals and the block's weights random codes.
"""
from __future__ import annotations

import argparse
import random

import torch

import mxfp4_mixture_experts_route_gb300 as moe


class VerifyStep:
    """A batch of B requests of up to n drafted tokens each, `layers` layers with a K/V cache each."""

    def __init__(self, B=4, n=8, layers=2, Hq=32, Hkv=8, D=128, page=64, most_ctx=4096, E=16, k=4, I=256, e4m3=False,
                 seed=0, projections=False, H=1024):
        self.B, self.n, self.layers, self.page = B, n, layers, page
        T = self.T = B * n
        gen = torch.Generator("cuda").manual_seed(seed)
        self.gen, self.pick = gen, random.Random(seed)
        width = -(-(most_ctx + n) // page)
        n_pages = B * width
        words = -(-n // 32)
        self.shape = moe.KVShape.of(B, T, Hq, Hkv, D, page, n_pages, width, mask_words=words, e4m3=e4m3)
        self.kv_ws = moe.new_kv_workspace(self.shape)

        def i32(*size):
            return torch.zeros(size, dtype=torch.int32, device="cuda")

        # what the host writes before a step, and what the plan writes
        self.ctx, self.new, self.parents, self.free = i32(B), i32(B), i32(T), i32(n_pages)
        self.table, self.row_start, self.positions, self.mask = i32(B, width), i32(B + 1), i32(T), i32(T, words)
        self.used, self.slots = i32(2), torch.zeros(T, dtype=torch.int64, device="cuda")
        self.accepted = torch.full_like(self.slots, -1)
        # the layers' caches and inputs
        dt = torch.uint8 if e4m3 else torch.bfloat16
        self.k_scale = self.v_scale = torch.full((Hkv,), 0.01, device="cuda") if e4m3 else None
        self.caches = [[torch.zeros(n_pages, Hkv, page, D, dtype=dt, device="cuda") for _ in "kv"] for _ in range(layers)]
        self.q = [torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(layers)]
        self.kv_new = [[torch.zeros(T, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in "kv"] for _ in range(layers)]
        self.attn = [torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(layers)]
        # the routed block of each layer, on the heads side by side
        d = Hq * D

        def codes(*size, low=0, high=256):
            return torch.randint(low, high, size, dtype=torch.uint8, device="cuda", generator=gen)

        block = moe.MoEShape.of(T, d, E, k, I)
        self.blocks = [moe.DeviceWeights(
            block, None, (torch.randn(E, d, device="cuda", generator=gen) * d ** -0.5).bfloat16(),
            torch.zeros(E, device="cuda"), None, codes(E, 2 * I, d // 2), codes(E, 2 * I, d // 32, low=119, high=121),
            codes(E, d, I // 2), codes(E, d, I // 32, low=121, high=123), None) for _ in range(layers)]
        self.projections = projections
        if projections:
            self._init_projections(H, most_ctx + n)
        # the host's own account of pages and lengths
        self.lens, self.pages, self.free_pages = [0] * B, [[] for _ in range(B)], list(range(n_pages))
        self.graph = None

    def _init_projections(self, H, max_pos):
        """The layers' input rows, their projections' weights (normal values, quantised) and what stands between."""
        T, Hq, Hkv, D = self.T, self.shape.Hq, self.shape.Hkv, self.shape.D
        width, d = (Hq + 2 * Hkv) * D, Hq * D

        def u8(*size):
            return torch.empty(size, dtype=torch.uint8, device="cuda")

        def weights(N, K):
            codes, scales = u8(N, K // 2), u8(N, K // 32)
            w = torch.randn(N, K, device="cuda", generator=self.gen) * K ** -0.5
            moe.mx_quantize(w.bfloat16(), codes, scales)
            return codes, scales

        self.x = [torch.zeros(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(self.layers)]
        self.w_qkv = [weights(width, H) for _ in range(self.layers)]
        self.w_o = [weights(d, d) for _ in range(self.layers)]
        self.norms = [[0.5 + torch.rand(D, device="cuda", generator=self.gen) for _ in "qk"] for _ in range(self.layers)]
        self.qkv = [torch.zeros(T, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(self.layers)]
        self.block_in = [torch.zeros(T, d, dtype=torch.bfloat16, device="cuda") for _ in range(self.layers)]
        self.rope_table = moe.rope_table(max_pos, D)
        self.rope = moe.Rope.of(D, max_pos, q_in_stride=width)
        # (the shape of the cache calls, K and V rows a projection's row apart)
        s = self.shape
        self.qkv_shape = moe.KVShape.of(s.B, s.T, Hq, Hkv, D, s.page, s.n_pages, s.max_pages, mask_words=s.W,
                                        e4m3=self.k_scale is not None, kv_stride=width)
        self.in_shape = moe.MXShape.of(T, width, H)
        self.out_shape = moe.MXShape.of(T, d, d, x_mxfp4=True)
        self.in_ws, self.out_ws = moe.new_mx_workspace(self.in_shape), moe.new_mx_workspace(self.out_shape)
        self.attn_codes, self.attn_scales = u8(T, d // 2), u8(T, d // 32)

    def _append_rows(self, layer, slots):
        """Norms, rotation and append of the layer's projected rows."""
        Hq, Hkv = self.shape.Hq, self.shape.Hkv
        rows = self.qkv[layer]
        moe.qkv_append(self.qkv_shape, self.rope, rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:], self.positions,
                       slots, *self.norms[layer], self.rope_table, self.k_scale, self.v_scale, self.q[layer],
                       *self.caches[layer], self.kv_ws)

    def _launch_projected(self):
        """With the projections: product, norms and append, attention, quantised rows, product and block in every layer."""
        for i, ((k, v), out, block) in enumerate(zip(self.caches, self.attn, self.blocks)):
            moe.mx_linear(self.in_shape, self.x[i], None, *self.w_qkv[i], self.qkv[i], self.in_ws)
            self._append_rows(i, self.slots)
            moe.tree_attention(self.shape, self.q[i], k, v, self.table, self.ctx, self.row_start, self.mask, self.k_scale,
                               self.v_scale, out, None, self.kv_ws)
            moe.mx_quantize(out.view(self.T, -1), self.attn_codes, self.attn_scales)
            moe.mx_linear(self.out_shape, self.attn_codes, self.attn_scales, *self.w_o[i], self.block_in[i], self.out_ws)
            block.forward(self.block_in[i])

    def launch(self):
        """The step's calls: 1 plan, then append, attention and block in every layer."""
        moe.kv_plan(self.shape, self.ctx, self.new, self.parents, self.free, self.table, self.row_start, self.slots,
                    self.positions, self.mask, self.used, self.kv_ws)
        if self.projections:
            return self._launch_projected()
        for q, (kn, vn), (k, v), out, block in zip(self.q, self.kv_new, self.caches, self.attn, self.blocks):
            moe.kv_append(self.shape, kn, vn, self.slots, self.k_scale, self.v_scale, k, v, self.kv_ws)
            moe.tree_attention(self.shape, q, k, v, self.table, self.ctx, self.row_start, self.mask, self.k_scale,
                               self.v_scale, out, None, self.kv_ws)
            block.forward(out.view(self.T, -1))

    def step(self, trees):
        """trees: a request's parents, drafted token by drafted token (-1: it follows the cache).  Returns ms."""
        news = [len(t) for t in trees]
        flat = [p for t in trees for p in t]
        self.ctx.copy_(torch.tensor(self.lens))
        self.new.copy_(torch.tensor(news))
        self.parents[:len(flat)] = torch.tensor(flat, dtype=torch.int32)
        # (-1 ends the list: the graph was captured with the length of the whole tensor)
        self.free.copy_(torch.tensor(self.free_pages + [-1] * (len(self.free) - len(self.free_pages)), dtype=torch.int32))
        for x in self.x if self.projections else (*self.q, *(t for kv in self.kv_new for t in kv)):
            x.normal_(generator=self.gen)
        if self.graph is None:
            self.launch()                        # (also the first step's work: a step may run twice)
            torch.cuda.synchronize()
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.launch()
        t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        t0.record()
        self.graph.replay()
        t1.record()
        for ws in (self.kv_ws, self.in_ws, self.out_ws) if self.projections else (self.kv_ws,):
            moe.check_device_status(ws, "verify step")
        for block in self.blocks:
            moe.check_device_status(block.ws, "verify step")
        # the pages the plan took, in its order
        for b, m in enumerate(news):
            need = -(-(self.lens[b] + m) // self.page) - len(self.pages[b])
            self.pages[b] += self.free_pages[:need]
            del self.free_pages[:need]
        return t0.elapsed_time(t1)

    def accept(self, paths):
        """paths: the accepted tokens of each request's tree, from a first one down.  Keeps their K and V only."""
        starts = self.row_start.tolist()
        slots, moved = self.slots.tolist(), [-1] * self.T
        for b, path in enumerate(paths):
            for i, token in enumerate(path):
                moved[starts[b] + token] = slots[starts[b] + i]
        self.accepted.copy_(torch.tensor(moved))
        for i, ((kn, vn), (k, v)) in enumerate(zip(self.kv_new, self.caches)):
            if self.projections:
                self._append_rows(i, self.accepted)
            else:
                moe.kv_append(self.shape, kn, vn, self.accepted, self.k_scale, self.v_scale, k, v, self.kv_ws)
        for b, path in enumerate(paths):
            self.lens[b] += len(path)
            keep = -(-self.lens[b] // self.page)
            self.free_pages += self.pages[b][keep:]
            del self.pages[b][keep:]

    def draft(self):
        """A random tree for each request, and a path down it."""
        trees, paths = [], []
        for _ in range(self.B):
            tree = [-1] + [self.pick.randrange(-1, i) for i in range(1, self.pick.randint(1, self.n))]
            path = [self.pick.randrange(len(tree))]
            while tree[path[0]] >= 0:
                path.insert(0, tree[path[0]])
            trees.append(tree)
            paths.append(path)
        return trees, paths


def main(argv=None):
    ap = argparse.ArgumentParser(prog="verify_step")
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--e4m3", action="store_true", help="an e4m3 cache")
    ap.add_argument("--projections", action="store_true", help="layers from their input rows, with MXFP4 projections")
    a = ap.parse_args(argv)
    s = VerifyStep(layers=a.layers, e4m3=a.e4m3, projections=a.projections)
    times = []
    for i in range(a.steps):
        trees, paths = s.draft()
        times.append(s.step(trees))
        s.accept(paths)
    times.sort()
    print(f"{a.steps} steps of {s.B} requests, {a.layers} layers: {times[len(times) // 2] * 1e3:.0f} us a step (median), "
          f"contexts {s.lens}, {s.shape.n_pages - len(s.free_pages)} pages held, "
          f"last plan: {s.used[0].item()} rows, {s.used[1].item()} pages")


if __name__ == "__main__":
    main()
