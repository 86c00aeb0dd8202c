"""One quantised expert layer, forward and backward: residual norm, products in NVFP4, gradients
in MXFP8.

    python examples/expert_layer.py [--experts 16] [--rows 4096] [--out 2048] [--cols 4096]

Forward: the residual's addition, the RMS norm and the NVFP4 encoding of the layer's input in one
call, then the product with each row's expert. Backward: the output's gradient goes to MXFP8
with stochastic rounding, by rows for the rows' gradient and by columns for the weights'; the
forward's encodings of the weights and of the input are de-quantised, transposed and encoded in
MXFP8 for them. Rows lie expert by expert; an expert's rows are padded with zeros to a multiple of 32.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import nvfp4_block_scaled_02_gb300 as nv  # noqa: E402

RNE = nv.Config()


class ExpertLayer:
    """Encoded weights [experts, out, cols] of a layer, its norm and its buffers. in_amax: the
    (calibrated) largest magnitude of the normed input."""

    def __init__(self, weights, norm_weight, in_amax=8.0, eps=1e-6):
        self.norm_weight, self.eps, dev = norm_weight, eps, weights.device
        self.amax = torch.full((1,), in_amax, device=dev)
        self.w_amax = nv.nvfp4_amax(weights)
        self.w = nv.nvfp4_quantize(weights, self.w_amax, RNE, dequant=False)["row"]
        # blocks along the rows' gradient's own sum: [experts, cols, out]
        self.wt = nv.nvfp4_requant_transpose(self.w["codes"], self.w["scales"], self.w_amax, RNE, RNE)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.products = nv.grouped_matmul_workspace(dev)
        self.norms = nv.add_rms_norm_workspace(dev)

    def forward(self, x, residual, start):
        """bf16 [rows, out], and what the backward pass needs."""
        n = nv.nvfp4_add_rms_norm(x, self.norm_weight, residual, eps=self.eps,
                                  global_amax=self.amax, status=self.status)
        y = nv.nvfp4_grouped_matmul(n, self.amax, self.w, self.w_amax, start,
                                    workspace=self.products, status=self.status)
        return y, n

    def backward(self, gy, n, start, gh=None, step=0):
        """Gradients of x (and of the residual), of every expert's weights (fp32) and of the
        norm's weight, from the output's gradient and, where the residual stream goes on, h's."""
        g = nv.nvfp4_mx_quantize(gy, nv.Config(blocks=nv.BLOCKS_BOTH, rounding=nv.ROUND_SR,
                                               step=step), status=self.status)
        xt = nv.nvfp4_requant_transpose(n["codes"], n["scales"], self.amax, RNE, RNE,
                                        status=self.status)
        gn = nv.nvfp4_mx_grouped_matmul(g["row"], self.wt, start, workspace=self.products,
                                        status=self.status)
        gw = nv.nvfp4_mx_grouped_wgrad(g["col"], xt, start, out_dtype=torch.float32,
                                       workspace=self.products, status=self.status)
        r = nv.nvfp4_add_rms_norm_bwd(gn, n["h"], self.norm_weight, gh, eps=self.eps,
                                      workspace=self.norms, status=self.status)
        return {"x": r["gx"], "weights": gw, "norm_weight": r["gw"], "encoded": (g, xt, gn)}


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--rows", type=int, default=4096)
    ap.add_argument("--out", type=int, default=2048)
    ap.add_argument("--cols", type=int, default=4096)
    a = ap.parse_args()
    torch.manual_seed(0)

    def randn(*shape, size=1.0):
        return (torch.randn(*shape, device="cuda") * size).to(torch.bfloat16)

    layer = ExpertLayer(randn(a.experts, a.out, a.cols, size=a.cols ** -0.5),
                        torch.ones(a.cols, dtype=torch.bfloat16, device="cuda"))
    rows = a.rows // 32 * 32
    cut = torch.sort(torch.randint(0, rows // 32 + 1, (a.experts - 1,))).values * 32
    start = torch.cat([torch.tensor([0]), cut, torch.tensor([rows])]).int().cuda()
    x, res, gy, gh = (randn(rows, a.cols), randn(rows, a.cols), randn(rows, a.out, size=1e-2),
                      randn(rows, a.cols, size=1e-2))

    def step():
        y, n = layer.forward(x, res, start)
        return y, layer.backward(gy, n, start, gh)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, g = step()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    graph.replay()
    begin.record()
    for _ in range(10):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    us = begin.elapsed_time(end) * 100
    flops = 6 * rows * a.out * a.cols
    print(f"{a.experts} experts, {rows} rows: {us:.1f} us a step (forward and backward, "
          f"{flops / us / 1e6:.0f} TFLOP/s), status {int(layer.status.item())}, output "
          f"{tuple(y.shape)}, weights' gradient {tuple(g['weights'].shape)}")


if __name__ == "__main__":
    main()
