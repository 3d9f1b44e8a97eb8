"""Calls of the operators of include/tsenor_ops.h that the binding refuses by itself, before the library is
called: arguments, the type of the error and what its message says.  Imported by tests only."""
import torch


def calls(device, sms):
    """(name, function's name, arguments, named arguments, error, message)."""
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32

    def new(*shape, dtype=bf16):
        return torch.zeros(*shape, dtype=dtype, device=device)

    # (two operands that share bytes come from one buffer)
    x, w, dy, ends = new(40, 32), new(4, 64, 32), new(40, 64), new(4, dtype=i32)
    y, dw, mask = new(40, 64), new(4, 64, 32), new(4, 64, 1, dtype=i32)
    q = sms.DenseInt8(new(40, 128, dtype=torch.int8), new(40, dtype=f32), 32)
    a = sms.DenseInt8(new(64, 128, dtype=torch.int8), new(64, dtype=f32), 32)
    ae = sms.DenseInt8(new(4, 64, 128, dtype=torch.int8), new(4, 64, dtype=f32), 32)
    wide = new(40, 200)
    g, m = new(4, 40, dtype=f32), new(4, 2, dtype=i32)
    h, shared = g.clone(), new(168, dtype=f32)
    over, over_mask = shared[:160].view(4, 40), shared[156:164].view(i32).view(4, 2)
    V, T = ValueError, TypeError
    return [
        # products
        ("X not bf16", "grouped_mm", (x.float(), w, ends), {}, T, "X must be bfloat16"),
        ("X of 1 dimension", "grouped_mm", (x[0], w, ends), {}, V, "X must be 2-D"),
        ("X of strided columns", "grouped_mm", (x.t(), w, ends), {}, V, "X must be 2-D with unit column stride"),
        ("W not bf16", "grouped_mm", (x, w.float(), ends), {}, T, "W must be bfloat16"),
        ("W of 2 dimensions", "grouped_mm", (x, w[0], ends), {}, V, "W must be 3-D"),
        ("W of strided columns", "grouped_mm", (dy, w.transpose(1, 2), ends), {}, V, "W must be 3-D with unit column stride"),
        ("W of fewer columns", "grouped_mm", (x, w[:, :, :-1], ends), {}, V, "X has 32 columns, W needs 31"),
        ("W transposed of fewer rows", "grouped_mm", (dy, w[:, :-1], ends), dict(transpose=True), V, "X has 64 columns, W needs 63"),
        ("fewer ends", "grouped_mm", (x, w, ends[:-1]), {}, V, "ends must be"),
        ("64-bit ends", "grouped_mm", (x, w, ends.long()), {}, V, "ends must be"),
        ("strided ends", "grouped_mm", (x, w, new(8, dtype=i32)[::2]), {}, V, "ends must be"),
        ("ends of 2 dimensions", "grouped_mm", (x, w, ends.view(2, 2)), {}, V, "ends must be"),
        ("ends no tensor", "grouped_mm", (x, w, [40] * 4), {}, V, "ends must be"),
        ("out of fewer rows", "grouped_mm", (x, w, ends), dict(out=y[:-1]), V, r"out must be a tensor of shape \(40, 64\)"),
        ("out of strided columns", "grouped_mm", (x, w, ends), dict(out=new(64, 40).t()), V, "out must be 2-D with unit column stride"),
        ("out of one place", "grouped_mm", (x, w, ends), dict(out=y.view(-1)[:1].expand(40, 64)), V, "out must be 2-D with unit column stride"),
        ("out whose rows overlap", "grouped_mm", (x, w, ends), dict(out=y.as_strided((40, 64), (63, 1))), V, "the rows of out overlap"),
        ("out of another type", "grouped_mm", (x, w, ends), dict(out=y, dtype=f32), V, "type torch.float32"),
        ("out in fp16", "grouped_mm", (x, w, ends), dict(out=y.half()), T, "out must be float32 or bfloat16"),
        ("result in fp16", "grouped_mm", (x, w, ends), dict(dtype=torch.float16), T, "out must be float32 or bfloat16"),
        ("out over X", "grouped_mm", (wide[:, :32], w, ends), dict(out=wide[:, 31:95]), V, "out overlaps an input"),
        ("out over W", "grouped_mm", (x, w, ends), dict(out=w.view(-1)[:2560].view(40, 64)), V, "out overlaps an input"),
        ("out over ends", "grouped_mm", (x, w, y.view(-1).view(i32)[8:12]), dict(out=y), V, "out overlaps an input"),
        ("X without columns", "grouped_mm", (x[:, :0], w[:, :, :0], ends), {}, V, "X has no columns"),
        ("transposed, X without columns", "grouped_mm", (x[:, :0], w[:, :0], ends), dict(transpose=True), V, "X has no columns"),
        ("no expert", "grouped_mm", (x, w[:0], ends[:0]), {}, V, "W holds no expert"),
        # weight gradients
        ("dY not bf16", "grouped_wgrad", (dy.float(), x, ends), {}, T, "dY must be bfloat16"),
        ("dY of fewer rows", "grouped_wgrad", (dy[:-1], x, ends), {}, V, "dY has 39 rows, X has 40"),
        ("64-bit ends", "grouped_wgrad", (dy, x, ends.long()), {}, V, r"ends must be a contiguous int32 tensor of shape \[experts\]"),
        ("a mask of more words", "grouped_wgrad", (dy, x, ends), dict(mask=new(4, 64, 2, dtype=i32)), V, "mask must be a contiguous"),
        ("a mask of fewer experts", "grouped_wgrad", (dy, x, ends), dict(mask=mask[:3]), V, "mask must be a contiguous"),
        ("a mask of 64-bit words", "grouped_wgrad", (dy, x, ends), dict(mask=mask.long()), V, "mask must be a contiguous"),
        ("a strided mask", "grouped_wgrad", (dy, x, ends), dict(mask=new(4, 64, 2, dtype=i32)[..., ::2]), V, "mask must be a contiguous"),
        ("out of fewer experts", "grouped_wgrad", (dy, x, ends), dict(out=dw[:3]), V, r"out must be a tensor of shape \(4, 64, 32\)"),
        ("out of more columns", "grouped_wgrad", (dy, x, ends), dict(out=new(4, 64, 33)), V, "out must be a tensor of shape"),
        ("out of another type", "grouped_wgrad", (dy, x, ends), dict(out=new(4, 64, 32, dtype=f32), dtype=bf16), V, "type torch.bfloat16"),
        ("out whose rows overlap", "grouped_wgrad", (dy, x, ends), dict(out=dw.as_strided((4, 64, 32), (2048, 31, 1))), V, "the rows of out overlap"),
        ("out whose matrices overlap", "grouped_wgrad", (dy, x, ends), dict(out=dw.as_strided((4, 64, 32), (2047, 32, 1))), V, "the matrices of out overlap"),
        ("out over dY", "grouped_wgrad", (dw.view(-1)[:2560].view(40, 64), x, ends), dict(out=dw), V, "out overlaps an input"),
        ("out over the mask", "grouped_wgrad", (dy, x, ends), dict(mask=dw.view(-1).view(i32)[:256].view(4, 64, 1), out=dw), V, "out overlaps an input"),
        # integers
        ("X of 1 dimension", "quant_int8", (x[0],), {}, V, "X must be 2-D"),
        ("X in fp16", "quant_int8", (x.half(),), {}, T, "X must be float32 or bfloat16"),
        ("X without columns", "quant_int8", (x[:, :0],), {}, V, "X has no columns"),
        ("X of 4 dimensions", "quant_int8", (new(2, 2, 2, 8),), {}, V, "X must be 2-D"),
        ("A no operand", "gemm_int8", (x, w[0]), {}, T, "A must be a DenseInt8 operand"),
        ("A a stack without ends", "gemm_int8", (x, ae), {}, V, "A.values must have 2 dimensions"),
        ("A no stack with ends", "gemm_int8", (x, a), dict(ends=ends), V, "A.values must have 3 dimensions"),
        ("A of fewer experts", "gemm_int8", (x, ae), dict(ends=ends[:3]), V, "A.values must be a contiguous"),
        ("A of another k", "gemm_int8", (x[:, :-1], a), {}, V, "X has 31 columns, A has 32"),
        ("A of a k past its columns", "gemm_int8", (x, a._replace(k=129)), {}, V, "A.values must be a contiguous"),
        ("A's scales too few", "gemm_int8", (x, a._replace(scales=a.scales[:-1])), {}, V, "A.scales must be a contiguous"),
        ("A's scales in bf16", "gemm_int8", (x, a._replace(scales=a.scales.to(bf16))), {}, V, "A.scales must be a contiguous"),
        ("A's values of another type", "gemm_int8", (x, a._replace(values=a.values.to(torch.uint8))), {}, V, "A.values must be a contiguous"),
        ("A's values strided", "gemm_int8", (x, a._replace(values=new(64, 256, dtype=torch.int8)[:, :128])), {}, V, "A.values must be a contiguous"),
        ("X's scales too few", "gemm_int8", (q._replace(scales=q.scales[1:]), a), {}, V, "X.scales must be a contiguous"),
        ("X in fp16", "gemm_int8", (x.half(), a), {}, T, "X must be float32 or bfloat16"),
        ("out over A's values", "gemm_int8", (x, a), dict(out=a.values.view(-1)[:5120].view(bf16).view(40, 64)), V, "out overlaps an input"),
        ("out over A's scales", "gemm_int8", (x, a._replace(scales=y.view(-1).view(f32)[4:68])), dict(out=y), V, "out overlaps an input"),
        ("out over X's scales", "gemm_int8", (q._replace(scales=y.view(-1).view(f32)[4:44]), a), dict(out=y), V, "out overlaps an input"),
        ("out of fewer columns", "gemm_int8", (x, a), dict(out=y[:, 1:]), V, r"out must be a tensor of shape \(40, 64\)"),
        ("X without columns", "gemm_int8", (x[:, :0], sms.DenseInt8(a.values[:, :0], a.scales, 0)), {}, V, "X has no columns"),
        ("integers without columns", "gemm_int8", (sms.DenseInt8(q.values[:, :0], q.scales, 0), sms.DenseInt8(a.values[:, :0], a.scales, 0)), {}, V, "X has no columns"),
        ("no expert", "gemm_int8", (x, sms.DenseInt8(ae.values[:0], ae.scales[:0], 32)), dict(ends=ends[:0]), V, "A holds no expert"),
        # gradients
        ("a gradient twice", "clip_grads", ([x, x], 1.0), {}, V, "a gradient that is written overlaps"),
        ("a gradient and rows of it", "clip_grads", ([x, x[3:5]], 1.0), {}, V, "a gradient that is written overlaps"),
        ("out over another gradient", "clip_grads", ([g, h], 1.0), dict(out=[h, new(4, 40, dtype=f32)]), V, "a gradient that is written overlaps"),
        ("out over a mask", "clip_grads", ([g], 1.0), dict(masks=[over_mask], out=[over]), V, "a gradient that is written overlaps"),
        ("fewer masks", "clip_grads", ([g], 1.0), dict(masks=[]), V, "masks must hold one entry"),
        ("fewer outs", "clip_grads", ([g], 1.0), dict(out=[]), V, "out must hold one tensor"),
        ("a mask of fewer words", "clip_grads", ([g], 1.0), dict(masks=[m[:, :1]]), V, r"masks\[0\] must be a contiguous int32"),
        ("a mask of 64-bit words", "grad_norm", ([g],), dict(masks=[m.long()]), V, r"masks\[0\] must be a contiguous int32"),
        ("out of another shape", "clip_grads", ([g], 1.0), dict(out=[g[:3].clone()]), V, r"out\[0\] must be a tensor like"),
        ("out of another type", "clip_grads", ([g], 1.0), dict(out=[g.to(bf16)]), V, r"out\[0\] must be a tensor like"),
        ("a strided gradient", "grad_norm", ([new(4, 4, 80)[..., ::2]],), {}, V, r"grads\[0\] must be contiguous"),
        ("a turned gradient under a mask", "grad_norm", ([new(40, 4, dtype=f32).t()],), dict(masks=[m]), V, r"grads\[0\] must be contiguous"),
        ("a gradient in fp64", "clip_grads", ([g.double()], 1.0), {}, T, r"grads\[0\] must be float32 or bfloat16"),
        ("no tensor in the list", "clip_grads", ([g, None], 1.0), {}, T, r"grads\[1\] must be a tensor"),
    ]
