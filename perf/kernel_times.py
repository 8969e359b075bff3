"""Device time of the operators' calls, without the host's share of a call.

    python perf/kernel_times.py [PREFIX ...]     cases whose names start so; all by default

Each case is prepared from three seeds and captured into a CUDA graph of many calls that take
the three states in turn; the figure is the median over replays of a replay's time by the number
of calls.  Three states of the larger cases exceed L2; those of the smaller ones stay in it, as
they do between the calls of a model.  Beside the cases of ``operators.py`` stand variants of
them: other sizes, and the parts of the product's epilogue one by one.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import operators  # noqa: E402


def cases():
    c = {x["name"]: x for x in operators.listed()}
    norm, grad, wide = c["norm_train"], c["norm_grad_train"], c["norm_grad_wide"]
    gate, down, odd, act = c["mm_gate_train"], c["mm_down_train"], c["mm_ragged"], c["act_grad_gated"]
    bias, token = c["act_grad_bias"], c["mm_one_token"]
    c.update({
        "norm_1537": dict(norm, cols=1537),
        "norm_4096x8192": dict(norm, rows=4096, cols=8192),
        "norm_fp32_8192x1536": dict(norm, dtype="fp32"),
        "norm_fp32_4096x8192": dict(norm, rows=4096, cols=8192, dtype="fp32"),
        "norm_fp32_2048x12288": dict(norm, rows=2048, cols=12288, dtype="fp32"),
        "norm_grad_1537": dict(grad, cols=1537),
        "norm_grad_128x1536": dict(grad, rows=128),
        "norm_grad_fp32_2048x12288": dict(wide, cols=12288, dres=True),
        "act_grad_gated_db": dict(act, db=True),
        "act_grad_gated_512_db": dict(act, rows=512, db=True),
        "act_grad_gated_1537_db": dict(act, cols=1537, db=True),
        "act_grad_bias_8192": dict(bias, rows=8192),
        "act_grad_fp32_8192_db": dict(c["act_grad_ragged"], rows=8192, cols=4096),
    })
    for k in (128, 1536):  # with K = 128 the products are a twelfth of the case's
        c["mm_gate_k%d" % k] = dict(gate, K=k)
        c["mm_gate_k%d_no_aux" % k] = dict(gate, K=k, aux="none")
        c["mm_gate_k%d_no_z" % k] = dict(gate, K=k, z=False)
        c["mm_gate_k%d_codes" % k] = dict(gate, K=k, aux="none", z=False)
        c["mm_gate_k%d_bf16" % k] = dict(gate, K=k, aux="none", z=False, act="none", out="bf16")
    for n in (1536, 1537, 1544):
        for z, out in ((False, "bf16"), (True, "bf16"), (False, "e4m3"), (True, "e4m3")):
            c["mm_odd_%d_%s%s" % (n, out, "_z" if z else "")] = dict(odd, N=n, z=z, out=out)
    for m in (1, 8, 16, 24, 64, 128, 256, 512):
        c["mm_rows_%d_4096x1536" % m] = dict(token, M=m)
        c["mm_rows_%d_1536x4096" % m] = dict(down, M=m)
    return c


def device_us(case, replays=9):
    states = [operators.prepare(case, seed) for seed in range(3)]
    for s in states:
        operators.run(s)
    calls = 12 if operators.work(case)["bytes"] > 5e7 else 48
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(calls):
            operators.run(states[i % 3])
    times = []
    for _ in range(replays):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        graph.replay()
        start.record()
        graph.replay()
        end.record()
        torch.cuda.synchronize()
        times.append(start.elapsed_time(end) * 1e3 / calls)
    return sorted(times)[replays // 2]


def main():
    operators.own = True
    wanted = tuple(sys.argv[1:])
    for name, case in cases().items():
        if wanted and not name.startswith(wanted):
            continue
        us, work = device_us(case), operators.work(case)
        print("%-28s %8.2f us %7.0f GB/s %7.0f TFLOP/s" % (name, us, work["bytes"] / us / 1e3, work["flops"] / us / 1e6),
              flush=True)


if __name__ == "__main__":
    main()
