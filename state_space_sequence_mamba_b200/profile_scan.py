"""Runs the prefill scan on one of the seeded workloads a few times and checks its status,
for a profiler to capture one launch of it:

    python -m state_space_sequence_mamba_b200.profile_scan CONFIG CHUNK REPS
    python -m state_space_sequence_mamba_b200.profile_scan bwd CONFIG REPS [fp32]
    python -m state_space_sequence_mamba_b200.profile_scan linattn|linattn_bwd REPS
    python -m state_space_sequence_mamba_b200.profile_scan group_norm|group_norm_bwd REPS

CONFIG is a workload of ``inputs.CONFIGS`` (1: SISO b4 L2048, 2: MIMO R4 b4 L2048, 4: b1
L65536), CHUNK the chunk length (64 / R for the 64-row tensor-core scan, 128 / R for the
128-row one), REPS the number of calls; BC normalisation is on. With ``bwd`` it runs the
backward (m3_scan_bwd) of the workload with its carried initial state and a seeded dy, in
the form the call picks, or the fp32 sweeps with ``fp32``. ``linattn`` and ``linattn_bwd``
run linear attention on 4 x 2048 tokens of 64 heads (K 128, V 64, bf16) and its gradients,
``group_norm`` and ``group_norm_bwd`` the centred and gated norm of 8192 rows of 4096 bf16
channels in groups of 64. Prints ``ok``."""
from __future__ import annotations

import sys


def main(argv=None) -> None:
    import torch
    from . import binding as m3
    from .inputs import make_config
    args = list(sys.argv[1:] if argv is None else argv)
    if args and args[0] == "bwd":
        backward(int(args[1]) if len(args) > 1 else 1, int(args[2]) if len(args) > 2 else 3,
                 len(args) > 3 and args[3] == "fp32")
        return
    if args and args[0] in ("linattn", "linattn_bwd", "group_norm", "group_norm_bwd"):
        operator(args[0], int(args[1]) if len(args) > 1 else 3)
        return
    cfg = int(args[0]) if args else 1
    chunk = int(args[1]) if len(args) > 1 else 64
    reps = int(args[2]) if len(args) > 2 else 3
    dev = torch.device("cuda:0")
    t = make_config(cfg).to(dev).tensors()
    dims = m3.make_dims(t["x"], t["B"], chunk, True, 1e-6, 0)
    ws = torch.zeros(m3.scan_workspace_bytes(dims), dtype=torch.uint8, device=dev)
    y = torch.empty_like(t["x"])
    for _ in range(reps):
        m3.scan_fwd(**t, chunk=chunk, bc_norm=True, y=y, workspace=ws)
    torch.cuda.synchronize()
    m3.scan_check(ws)
    print("ok")


def backward(cfg: int, reps: int, fp32: bool) -> None:
    import torch
    from . import binding as m3
    from .inputs import make_config
    dev = torch.device("cuda:0")
    pr = make_config(cfg, with_state=True).to(dev)
    g = torch.Generator(device=dev).manual_seed(cfg + 1)
    dy = torch.randn(pr.x.shape, generator=g, device=dev).to(pr.x.dtype)
    sa = pr.scalar_args()
    if fp32:
        sa["flags"] = sa["flags"] | m3.BWD_FP32
    dims = m3.make_dims(pr.x, pr.B, 1, pr.dims.bc_norm, pr.dims.norm_eps, sa["flags"])
    ws = torch.empty(m3.scan_bwd_workspace_bytes(dims), dtype=torch.uint8, device=dev)
    init = m3.State.from_dict(pr.state)
    for _ in range(reps):
        m3.scan_bwd(**pr.tensors(), dy=dy, init=init, bc_norm=pr.dims.bc_norm,
                    norm_eps=pr.dims.norm_eps, workspace=ws, **sa)
    torch.cuda.synchronize()
    m3.scan_check(ws)
    print("ok")


def operator(name: str, reps: int) -> None:
    import torch
    from . import binding as m3
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(1)

    def rand(*shape):
        return torch.randn(shape, generator=g, device=dev).to(torch.bfloat16)
    if name.startswith("linattn"):
        q, k, v, do = rand(4, 2048, 64, 128), rand(4, 2048, 64, 128), rand(4, 2048, 64, 64), rand(4, 2048, 64, 64)
        decay = torch.linspace(-0.5, -0.002, 64, device=dev)
        for _ in range(reps):
            if name == "linattn":
                m3.linattn_fwd(q, k, v, decay, scale=128 ** -0.5)
            else:
                m3.linattn_bwd(q, k, v, decay, do, scale=128 ** -0.5)
        torch.cuda.synchronize()
        m3.linattn_check()
    else:
        x, z, dout = rand(8192, 4096), rand(8192, 4096), rand(8192, 4096)
        w, b = torch.ones(4096, device=dev), torch.zeros(4096, device=dev)
        for _ in range(reps):
            if name == "group_norm":
                m3.group_norm_fwd(x, 64, w, b, z)
            else:
                m3.group_norm_bwd(dout, x, 64, w, b, z)
        torch.cuda.synchronize()
    print("ok")


if __name__ == "__main__":
    main()
