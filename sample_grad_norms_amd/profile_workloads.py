"""Runs one named workload a few times, for profiling with rocprofv3 (the
112-projection stack with independent inputs is profiled through bench.py).

    python sample_grad_norms_amd/profile_workloads.py NAME [--reps R] [--calib-copy] [--time]

NAME is one of:
  long_context_hutch  Hutchinson, B=1, T=32768, d=2048, p=8192, k=32
  long_context_exact  the exact explicit route on the same inputs
  hutchpp             Hutch++, B=4, T=4096, d=p=2048, budget 32
  single_layer        Hutchinson, B=8, T=1024, d=p=2048, k=32
  single_layer_gram   the exact Gram route on the same inputs
  shared_stack        the Llama-3.2-1B-shaped stack with q/k/v and gate/up
                      sharing their input (grouped Hutchinson, B=4, T=4096, k=32)
  sign_stack          the stack with +-1 projections stored as bits
  lora_routed         rank-16 LoRA factors of the stack, routed call (exact norms)
  dpsgd_step          DP-SGD-RC training steps on a random-init Llama-width stack
                      (2 decoder layers, B=4, T=2048, bf16): forward, backward 1,
                      the norm path, backward 2 of sum c_i l_i, noise, Adam
  dpsgd_step_library  the same with the library's attention
  dpsgd_step_tokens   the same from token ids, with the library's embedding table
                      (32768 rows, trained) and attention
  dpsgd_step_norms    dpsgd_step_library with the library's layer norms, trained, and
                      attention scores capped by a tanh and biased by distance
  embedding           lookup, order, per-sample norm and table gradient, B=4, T=4096,
                      d=2048, 131072 rows, ids by a vocabulary's frequencies, bf16
  attention           causal attention and its gradients, B=4, T=2048, 32 heads over
                      8, head width 64, bf16
  attention_capped, attention_biased, attention_prefix
                      the same with scores capped at 50, with a bias by distance, and
                      with a prefix of two fifths of each sample
  layernorm           layer norm's forward pass, gradients and per-sample norms, B=4,
                      T=4096, d=2048, bf16
--calib-copy first runs one 1 GiB device-to-device copy, the reference the
counter summaries scale FETCH_SIZE and WRITE_SIZE by. --time (for runs without
the profiler) prints the wall time of a call, after three that are not timed, and
the largest amount of memory allocated in them.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

NAMES = ("long_context_hutch", "long_context_exact", "hutchpp", "single_layer", "single_layer_gram", "shared_stack",
         "sign_stack", "lora_routed", "dpsgd_step", "dpsgd_step_library", "dpsgd_step_tokens", "dpsgd_step_norms",
         "embedding", "attention", "attention_capped", "attention_biased", "attention_prefix", "layernorm")


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("name", choices=NAMES)
    ap.add_argument("--reps", type=int, default=5)
    ap.add_argument("--calib-copy", action="store_true")
    ap.add_argument("--time", action="store_true")
    a = ap.parse_args()
    import torch
    import sample_grad_norms_amd as dp
    import workloads
    dev = torch.device("cuda:0")
    if a.calib_copy:
        src = torch.empty(1 << 30, dtype=torch.uint8, device=dev)
        torch.empty_like(src).copy_(src)
        torch.cuda.synchronize()
        del src
    if a.name.startswith("long_context"):
        pr = workloads.config5(device=dev)
        fn = (lambda: dp.hutch(pr.A, pr.G, pr.P)) if a.name.endswith("hutch") else (lambda: dp.exact(pr.A, pr.G))
    elif a.name == "hutchpp":
        pr = workloads.config4(device=dev)
        fn = lambda: dp.hutchpp(pr.A, pr.G, pr.S, pr.P, k=pr.k)
    elif a.name == "shared_stack":
        layers = workloads.shared_input_stack(device=dev)
        fn = lambda: dp.hutch_grouped(layers, C_clip=1.0)
    elif a.name == "sign_stack":
        projs = [workloads.config3_projection(j, device=dev) for j in range(112)]
        gen = torch.Generator(device=dev)
        gen.manual_seed(2024)
        triples = [(q.A, q.G, dp.random_signs(q.G.shape[2], 32, device=dev, generator=gen)) for q in projs]
        fn = lambda: dp.hutch_sign_grouped(triples, 32, C_clip=1.0)
    elif a.name == "lora_routed":
        routed = [(A, G, None) for (A, G, _) in workloads.lora_stack(device=dev)]
        fn = lambda: dp.norms_routed(routed, 32)
    elif a.name.startswith("dpsgd_step"):
        from sample_grad_norms_amd.dpsgd_rc import RandomizedClipping
        from workloads import llama_block as lb
        shape = dict(layers=2, dim=2048, heads=32, kv_heads=8, hidden=8192, vocab=2048)
        if a.name == "dpsgd_step_tokens":   # from token ids, with the library's table
            shape.update(vocab_in=32768, embed_scale=45.0)
        if a.name != "dpsgd_step":
            shape.update(ops="library")
        if a.name == "dpsgd_step_norms":
            shape.update(norm="layer", cap=50.0, distance=True)
        model = lb.build(90, device=dev, dtype=torch.bfloat16, **shape)
        x, y = lb.batch(91, 4, 2048, shape["dim"], shape["vocab"], device=dev, dtype=torch.bfloat16)
        if a.name == "dpsgd_step_tokens":
            x, y = lb.token_batch(91, 4, 2048, shape["vocab_in"], shape["vocab"], device=dev)
        rc = RandomizedClipping(model, C=1.0, noise_multiplier=1.0, k=32)
        opt = torch.optim.Adam(rc.params, lr=1e-5)

        def fn():
            with rc.capture():
                losses = lb.per_sample_loss(model(x), y)
            n, c = rc.clip_factors(losses)
            rc.clipped_backward(losses, c)
            rc.add_noise()
            opt.step()
            opt.zero_grad(set_to_none=True)
    elif a.name == "embedding":
        from workloads import llama_block as lb
        g = torch.Generator().manual_seed(92)
        tok, _ = lb.token_batch(93, 4, 4096, 131072, 2, device=dev)
        W = torch.randn(131072, 2048, generator=g).to(dev, torch.bfloat16)
        G = torch.randn(4, 4096, 2048, generator=g).to(dev, torch.bfloat16)
        c = torch.full((4,), 0.5, device=dev)

        def fn():
            dp.embed_lookup(tok, W)
            order = dp.embed_order(tok, 131072)
            dp.embed_norm(order, G)
            dp.embed_grad(order, G, weights=c)
    elif a.name == "layernorm":
        g = torch.Generator().manual_seed(95)
        x, G = (torch.randn(4, 4096, 2048, generator=g).to(dev, torch.bfloat16) for _ in range(2))
        w, b = (torch.randn(2048, generator=g).to(dev, torch.bfloat16) for _ in range(2))
        c = torch.full((4,), 0.5, device=dev)

        def fn():
            _, mean, rstd = dp.layernorm_forward(x, w, b)
            dp.layernorm_backward(G, x, w, mean, rstd, weights=c)
            dp.layernorm_norm(x, G)
    elif a.name.startswith("attention"):
        g = torch.Generator().manual_seed(94)
        q, do = (torch.randn(8192, 32, 64, generator=g).to(dev, torch.bfloat16) for _ in range(2))
        k, v = (torch.randn(8192, 8, 64, generator=g).to(dev, torch.bfloat16) for _ in range(2))

        how = {"attention": {}, "attention_capped": dict(cap=50.0),
               "attention_biased": dict(slopes=torch.exp2(-8.0 * torch.arange(1, 33) / 32).to(dev)),
               "attention_prefix": dict(prefix=torch.full((4,), 819, dtype=torch.int32, device=dev))}[a.name]

        def fn():
            o, lse = dp.attention_forward(q, k, v, sequences=4, **how)
            dp.attention_backward(do, q, k, v, o, lse, sequences=4, **how)
    else:
        pr = workloads.config2(device=dev)
        fn = (lambda: dp.exact(pr.A, pr.G, route="gram")) if a.name.endswith("gram") else (lambda: dp.hutch(pr.A, pr.G, pr.P))
    if a.time:
        for _ in range(3):
            fn()
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
    start = time.perf_counter()
    for _ in range(a.reps):
        fn()
    torch.cuda.synchronize()
    if a.time:
        print(f"{a.name}: {(time.perf_counter() - start) / a.reps * 1e3:.2f} ms a call, "
              f"{torch.cuda.max_memory_allocated() / 1e9:.2f} GB at most", flush=True)
    print(f"{a.name}: {a.reps} calls done", flush=True)


if __name__ == "__main__":
    main()
