"""The debug build's device-side checks in the attention of a training step: on
correct inputs none fires and every result equals the normal build's bit for
bit. Each build runs in a child process of its own."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import sys, torch
import tensor_transformer_mlp_column_gb300 as tp
torch.cuda.set_device(0)
assert bool(tp.tpmlp_build_flags() & 1) == (sys.argv[2] == "debug")
out = {}
cases = [  # lengths, rows behind them, heads, kv heads, head size, longest length stated, causal
    ([130, 1, 0, 77], 13, 4, 2, 64, None, True), ([130, 1, 0, 77], 13, 4, 2, 64, 130, False), ([300, 129], 0, 3, 1, 128, 300, True),
    ([40] * 70 + [513], 5, 2, 1, 72, None, True), ([1000], 0, 8, 1, 64, 1000, True), ([700, 1, 0, 300], 3, 16, 1, 128, 700, False),
    ([200, 200], 0, 4, 4, 40, 0, True),  # 0: equal sequences, without starts
]
for dt in (torch.bfloat16, torch.float32):
    for i, (lengths, behind, heads, kv, dim, most, causal) in enumerate(cases):
        g = torch.Generator(device="cuda").manual_seed(i)
        T = sum(lengths) + behind
        x = torch.randn(T, heads + 2 * kv, dim, generator=g, device="cuda").to(dt)
        do = torch.randn(T, heads, dim, generator=g, device="cuda").to(dt)
        w = (1 + 0.2 * torch.randn(dim, generator=g, device="cuda")).to(dt)
        q, k, v = x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]
        starts = torch.tensor([0] + lengths).cumsum(0).int().cuda()
        seqs = dict(batch=len(lengths)) if most == 0 else dict(starts=starts, max_seq=most)
        for inter in (False, True):
            rot = dim - 8 if inter else dim
            turn = dict(freqs=[10000.0 ** (-2 * j / rot) for j in range(rot // 2)], wq=w, wk=w, interleaved=inter)
            pos = torch.arange(T, device="cuda")
            yq, yk = tp.tpmlp_qk_rope_forward(q, k, pos, **turn)
            key = f"{dt}_{i}_{inter}_"
            o, lse = (torch.zeros_like(do), torch.zeros(heads, T, device="cuda"))
            tp.tpmlp_attn_core_forward(yq, yk, v, o=o, lse=lse, causal=causal, **seqs)
            d = torch.zeros_like(x)
            dq, dk, dv = d[:, :heads], d[:, heads:heads + kv], d[:, heads + kv:]
            tp.tpmlp_attn_core_backward(yq, yk, v, o, lse, do, dq=dq, dk=dk, dv=dv, causal=causal, **seqs)
            out[key + "d"] = d.clone()
            _, _, out[key + "dwq"], out[key + "dwk"] = tp.tpmlp_qk_rope_backward(dq, dk, q, k, pos, dq=dq, dk=dk, **turn)
            out.update({key + "yq": yq, key + "yk": yk, key + "o": o, key + "lse": lse, key + "dx": d})
            tp.tpmlp_check_status()
torch.cuda.synchronize()
torch.save({k: v.cpu() for k, v in out.items()}, sys.argv[1])
print("ok")
'''


def test_debug_build_matches_normal_build_in_the_attention_of_a_step(tmp_path):
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    from tensor_transformer_mlp_column_gb300 import build_lib

    __graft_entry__.build()
    build_lib.build(debug=True, quiet=True)
    results = {}
    for kind in ("debug", "normal"):
        path = str(tmp_path / f"{kind}.pt")
        env = dict(os.environ)
        env.pop("TPMLP_DEBUG", None)
        if kind == "debug":
            env["TPMLP_DEBUG"] = "1"
        r = subprocess.run([sys.executable, "-c", CHILD, path, kind], env=env, cwd=ROOT, capture_output=True,
                           text=True, timeout=900)
        assert r.returncode == 0 and r.stdout.strip().endswith("ok"), kind + r.stdout[-2000:] + r.stderr[-4000:]
        results[kind] = torch.load(path)
    assert results["debug"].keys() == results["normal"].keys()
    for k in results["normal"]:
        assert torch.equal(results["debug"][k], results["normal"][k]), f"{k}: debug and normal builds differ"
