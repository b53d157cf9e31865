"""The layer for a few tokens and its workspace, through the C ABI: whatever the
workspace holds (every byte value that could pass for a flag or a number, what
another call left), and calls that overlap, each in a workspace of its own that
still holds another input's rows.  Every pass is compared, bit for bit."""

import ctypes

import pytest
import torch

import sparse_moe_layer_latentmoe_amd as pkg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F, B = torch.float32, torch.bfloat16


class Call:
    """A layer with explicit workspaces."""

    def __init__(self, T, E, K, D, H, S, fmt, swiglu, out, xdtype):
        g = torch.Generator().manual_seed(T + E + D)

        def rand(*s, std=0.05):
            return (torch.randn(*s, generator=g) * std).to(DEV)

        def matrices(*s):
            w = rand(*s)
            if fmt == "bf16":
                return w.to(B), None
            return pkg.quantize_fp8_weight(w) if fmt == "fp8" else pkg.quantize_mxfp4(w.to(B))

        two = 2 if swiglu else 1
        self.T, self.K, self.D, self.out, self.xdtype = T, K, D, out, xdtype
        self.router = pkg.make_router(E, K)
        self.gate = rand(E, D, std=D ** -0.5)
        self.up, self.down = matrices(E, two * H, D), matrices(E, D, H)
        self.sh = (matrices(two * S, D), matrices(D, S)) if S else None
        self.g = g
        a = pkg.LmoeMoeTokensArgs()
        p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        a.router, a.x_stride, a.gate = self.router, D, p(self.gate)
        a.up, a.up_scales = p(self.up[0]), p(self.up[1])
        a.down, a.down_scales = p(self.down[0]), p(self.down[1])
        if S:
            (u, us), (d, ds) = self.sh
            a.shared_up, a.shared_up_scales = p(u), p(us)
            a.shared_down, a.shared_down_scales = p(d), p(ds)
        a.x_type, a.gate_type, a.y_type = int(xdtype == B), 0, int(out == B)
        a.expert_format = {"bf16": pkg.EXPERTS_BF16, "fp8": pkg.EXPERTS_FP8,
                           "mxfp4": pkg.EXPERTS_MXFP4}[fmt]
        a.activation = pkg.ACT_SWIGLU if swiglu else pkg.ACT_RELU2
        a.T, a.D, a.F, a.S = T, D, H, S
        self.a = a
        self.bytes = int(pkg.load_library().lmoe_moe_tokens_workspace_size(a))
        assert self.bytes > 0

    def input(self):
        return torch.randn(self.T, self.D, generator=self.g).to(self.xdtype).to(DEV)

    def outputs(self):
        return (torch.zeros(self.T, self.D, dtype=self.out, device=DEV),
                torch.zeros(self.T, self.K, dtype=torch.int32, device=DEV),
                torch.zeros(self.T, self.K, device=DEV))

    def __call__(self, x, ws, outputs=None, stream=0):
        o = self.outputs() if outputs is None else outputs
        a = pkg.LmoeMoeTokensArgs()
        ctypes.pointer(a)[0] = self.a
        a.x, a.y, a.topk_idx, a.topk_w = (t.data_ptr() for t in (x, *o))
        assert pkg.load_library().lmoe_moe_tokens(a, ws.data_ptr(), self.bytes,
                                                  stream) == pkg.LMOE_OK
        return o

    def workspace(self, byte=0):
        # (and a page behind it that must stay as it is)
        return torch.full((self.bytes + 4096,), byte, dtype=torch.uint8, device=DEV)


FORMS = [(1, 24, 4, 512, 384, 256, "bf16", False, B, F), (4, 300, 6, 256, 256, 0, "mxfp4", True, F, B),
         (8, 40, 5, 512, 256, 128, "fp8", True, B, B), (16, 6, 3, 384, 640, 384, "mxfp4", False, F, F),
         (13, 200, 8, 256, 320, 64, "bf16", True, B, B)]


def equal(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("form", FORMS)
def test_workspace_of_any_bytes(form):
    call = Call(*form)
    x, other = call.input(), call.input()
    want = call(x, call.workspace())
    assert all(bool(t.double().isfinite().all()) for t in want)
    for byte in (0xFF, 0x7F, 0x01, 0x80, 0x3F):
        ws = call.workspace(byte)
        assert equal(call(x, ws), want), byte
        assert bool((ws[call.bytes:] == byte).all())
        # what another input left, and the same one again
        call(other, ws)
        assert equal(call(x, ws), want)
        assert equal(call(x, ws), want)
    noise = torch.randint(0, 256, (call.bytes,), dtype=torch.uint8,
                          generator=torch.Generator().manual_seed(1)).to(DEV)
    assert equal(call(x, noise), want)


@pytest.mark.parametrize("form", FORMS)
def test_overlapping_calls_with_changing_inputs(form):
    call = Call(*form)
    xs = [call.input() for _ in range(5)]
    want = [call(x, call.workspace()) for x in xs]
    sides = [torch.cuda.Stream() for _ in range(4)]
    spaces = [call.workspace(0xFF) for _ in sides]
    # pass n of stream i takes input (n + i) % 5: never the one before
    outs = [[call.outputs() for _ in range(12)] for _ in sides]
    torch.cuda.synchronize()
    for n in range(12):
        for i, s in enumerate(sides):
            call(xs[(n + i) % 5], spaces[i], outs[i][n], s.cuda_stream)
    torch.cuda.synchronize()
    for i in range(4):
        for n in range(12):
            assert equal(outs[i][n], want[(n + i) % 5]), (i, n)
