"""Run a few decode steps of a workload, for profiling.

  python -m task_graph_runtime_gb300.run_steps --workload qwen3_8b \
      --mode mega --layers 1 --steps 3 [--coarse]
  python -m task_graph_runtime_gb300.run_steps --workload qwen3_8b_b16 \
      --mode verify --drafts 3 [--shared 2048]

Seeded synthetic weights and KV cache are generated on cuda:0; `--layers`
keeps only the first N decoder layers (a smaller case of the same kernels,
tiling and launch geometry, for profiler captures that must stay a few GB).
Every step rewinds the sequence lengths, so all steps do the same work.
Mode `verify` runs steps of drafted decoding (`Graph.verify_step`): the
workload's rows are the tokens of rows / (drafts + 1) sequences, `--shared`
makes them share their first tokens (at most the shortest context).
Prints the device memory in use and the mean step time (CUDA events)."""
from __future__ import annotations

import argparse
import dataclasses


def main():
    import torch

    from . import mpk, synth
    ap = argparse.ArgumentParser()
    ap.add_argument("--workload", default="qwen3_8b",
                    choices=sorted(synth.WORKLOADS))
    ap.add_argument("--mode", default="mega",
                    choices=["mega", "kpo", "kpo_graph", "verify"])
    ap.add_argument("--drafts", type=int, default=0,
                    help="mode verify: drafts of a sequence")
    ap.add_argument("--shared", type=int, default=0,
                    help="mode verify: tokens all sequences share")
    ap.add_argument("--layers", type=int, default=0,
                    help="keep the first N decoder layers (0: all)")
    ap.add_argument("--steps", type=int, default=3)
    ap.add_argument("--coarse", action="store_true",
                    help="operator-level events (the coarse-grained graph)")
    args = ap.parse_args()
    wl = synth.WORKLOADS[args.workload]
    s = wl.shape
    if args.layers > 0 and not s.is_chain:
        s = dataclasses.replace(s, n_layers=min(args.layers, s.n_layers))
        wl = dataclasses.replace(wl, shape=s)
    W = synth.device_model_weights(s, 0, "cuda")
    g = mpk.Graph(s, wl.batch, page_size=wl.page_size,
                  max_pages_per_seq=max(1, wl.max_pages_per_seq),
                  coarse_events=int(args.coarse))
    g.bind(mpk.Weights(W, s))
    if args.mode != "verify":
        g.set_mode({"mega": mpk.MODE_MEGAKERNEL, "kpo": mpk.MODE_KPO,
                    "kpo_graph": mpk.MODE_KPO_GRAPH}[args.mode])
    kv, seq0 = None, None
    if not s.is_chain:
        k, v, pt, sl = synth.device_kv_inputs(wl, 0, "cuda")
        seq0 = torch.from_numpy(sl).cuda()
        kv = mpk.KVCache(k, v, torch.from_numpy(pt).cuda(), seq0.clone())
    tok = torch.from_numpy(synth.tokens(wl, 0)).cuda()
    lg = torch.empty(wl.batch, s.vocab, device="cuda")
    nt = torch.empty(wl.batch, dtype=torch.int32, device="cuda")
    step = lambda: g.decode_step(tok, kv, lg, nt)
    if args.mode == "verify":
        rows = args.drafts + 1
        if s.is_chain or rows < 1 or wl.batch % rows:
            ap.error("mode verify needs a decoder whose batch is a multiple "
                     "of drafts + 1")
        n = wl.batch // rows
        kv = mpk.KVCache(kv.k_pool, kv.v_pool,
                         kv.page_table[:n].contiguous(),
                         (seq0 - args.drafts).clamp(min=0)[:n].contiguous())
        seq0 = kv.seq_lens.clone()
        groups = {}
        if args.shared:
            i32 = dict(dtype=torch.int32, device="cuda")
            groups = dict(group_start=torch.tensor([0, n], **i32),
                          prefix_len=seq0.min().clamp(max=args.shared).view(1))
        gen = torch.Generator(device="cuda").manual_seed(0)
        u = torch.rand(wl.batch, device="cuda", generator=gen)
        noise = torch.empty(n, s.vocab, device="cuda").exponential_(
            generator=gen)
        acc = torch.empty(n, dtype=torch.int32, device="cuda")
        out = torch.empty(n, rows, dtype=torch.int32, device="cuda")
        step = lambda: g.verify_step(tok, kv, lg, u, noise, acc, out,
                                     **groups)
    e0 = torch.cuda.Event(enable_timing=True)
    e1 = torch.cuda.Event(enable_timing=True)
    e0.record()
    for _ in range(args.steps):
        if kv is not None:
            kv.seq_lens.copy_(seq0)
        step()
    e1.record()
    torch.cuda.synchronize()
    if g.status() != mpk.MPK_OK:
        raise RuntimeError(mpk.STATUS_NAMES[g.status()])
    g.close()
    print(f"{args.workload} layers={s.n_layers} mode={args.mode}"
          f"{' coarse' if args.coarse else ''}: "
          f"{e0.elapsed_time(e1) / args.steps:.3f} ms/step, "
          f"{torch.cuda.memory_allocated() / 1e9:.2f} GB on the device")


if __name__ == "__main__":
    main()
