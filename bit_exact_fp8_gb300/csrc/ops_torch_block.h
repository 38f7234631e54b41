// ops_torch_block.h -- the operators of 8-bit layers with block scales on torch tensors (part of
// ops_torch.cpp, whose helpers it uses).
#pragma once

int64_t blocks_of(int64_t n) { return (n + 127) / 128; }

emu_fp8_t fp8_type(c10::ScalarType t, const char* name) {
  if (t == at::kFloat8_e4m3fn) return EMU_E4M3FN;
  if (t == at::kFloat8_e5m2) return EMU_E5M2;
  bad(std::string(name) + ": float8_e4m3fn or float8_e5m2 expected, got " + text(t));
}
emu_out_t out_type(c10::ScalarType t) {
  if (t != at::kFloat && t != at::kBFloat16 && t != at::kHalf) unsupported("out_dtype " + text(t) + " is not supported");
  return t == at::kFloat ? EMU_OUT_F32 : t == at::kBFloat16 ? EMU_OUT_BF16 : EMU_OUT_F16;
}
// a pair (rows, columns) that share a scale
emu_block_t block_shape(PyObject* o) {
  int64_t v[2] = {0, 0};
  if (PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 2)
    for (int i = 0; i < 2; ++i) v[i] = whole(PyTuple_GET_ITEM(o, i), "block");
  else
    throw Refused{PyExc_TypeError, "block must be a pair of whole numbers"};
  if (v[0] == 1 && v[1] == 128) return EMU_BLOCK_ROWS;
  if (v[0] == 128 && v[1] == 1) return EMU_BLOCK_COLUMNS;
  if (v[0] == 128 && v[1] == 128) return EMU_BLOCK_SQUARES;
  unsupported("block (" + std::to_string(v[0]) + ", " + std::to_string(v[1]) + "): (1, 128), (128, 1) and (128, 128) are supported");
}
at::Tensor block_scales(emu_block_t block, int64_t T, int64_t H, c10::Device dev) {
  return make({block == EMU_BLOCK_ROWS ? T : blocks_of(T), block == EMU_BLOCK_COLUMNS ? H : blocks_of(H)}, at::kFloat, dev);
}

// (x, block, out_dtype, out) -> (q, scale)
PyObject* block_quant(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "x");
  const c10::Device dev = first(x, "x");
  no_grad(x);
  const int64_t T = x.size(0), H = x.size(1);
  const emu_out_t type = float_type(x.scalar_type(), "x");
  const int64_t ldx = rows_of(x, "x", T, H, x.scalar_type(), dev);
  const emu_block_t block = block_shape(a[1]);
  const c10::ScalarType qt = dtype(a[2], "out_dtype");
  if (qt != at::kFloat8_e4m3fn && qt != at::kFloat8_e5m2) unsupported("out_dtype " + text(qt) + " is not supported");
  On on(dev);
  const at::Tensor q = a[3] == Py_None ? make({T, H}, qt, dev) : given(a[3], "out", T, H, qt, dev);
  const at::Tensor scale = block_scales(block, T, H, dev);
  check(emu_block_quant(x.data_ptr(), ldx, type, T, H, block, fp8_type(qt, "out_dtype"), q.data_ptr(), scale.data_ptr<float>(),
                        on.stream), "block_quant");
  if (a[3] != Py_None) written(q);
  return tuple_of({a[3] == Py_None ? THPVariable_Wrap(q) : same(a[3]), THPVariable_Wrap(scale)});
}

// (gate_up, block, out_dtype, checkpoint, out) -> (q, scale, checkpoint, checkpoint_scale)
PyObject* swiglu_quant(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "gate_up");
  const c10::Device dev = first(x, "gate_up");
  no_grad(x);
  const int64_t T = x.size(0), H = x.size(1) / 2;
  if (x.size(1) % 2) bad("gate_up: an even number of columns expected, got " + text(x));
  const emu_out_t type = float_type(x.scalar_type(), "gate_up");
  const int64_t ldx = rows_of(x, "gate_up", T, 2 * H, x.scalar_type(), dev);
  const emu_block_t block = block_shape(a[1]);
  if (block == EMU_BLOCK_COLUMNS) unsupported("block (128, 1): the output is quantised in (1, 128) or (128, 128)");
  const c10::ScalarType qt = dtype(a[2], "out_dtype");
  if (qt != at::kFloat8_e4m3fn && qt != at::kFloat8_e5m2) unsupported("out_dtype " + text(qt) + " is not supported");
  const int keep = PyObject_IsTrue(a[3]);
  if (keep < 0) {
    PyErr_Clear();
    throw Refused{PyExc_TypeError, "checkpoint must be true or false"};
  }
  On on(dev);
  const at::Tensor q = a[4] == Py_None ? make({T, H}, qt, dev) : given(a[4], "out", T, H, qt, dev);
  const at::Tensor scale = block_scales(block, T, H, dev);
  at::Tensor kept, kept_scale;
  if (keep) {
    kept = make({T, 2 * H}, at::kFloat8_e4m3fn, dev);
    kept_scale = make({T, 2 * blocks_of(H)}, at::kFloat, dev);
  }
  check(emu_swiglu_quant(x.data_ptr(), ldx, type, T, H, block, fp8_type(qt, "out_dtype"), q.data_ptr(), scale.data_ptr<float>(),
                         keep ? kept.data_ptr() : nullptr, keep ? kept_scale.data_ptr<float>() : nullptr, on.stream),
        "swiglu_quant");
  if (a[4] != Py_None) written(q);
  return tuple_of({a[4] == Py_None ? THPVariable_Wrap(q) : same(a[4]), THPVariable_Wrap(scale),
                   keep ? THPVariable_Wrap(kept) : same(Py_None), keep ? THPVariable_Wrap(kept_scale) : same(Py_None)});
}

// (grad_y, checkpoint, checkpoint_scale) -> grad_gate_up
PyObject* swiglu_backward(PyObject* const* a) {
  const at::Tensor& gy = tensor(a[0], "grad_y");
  const c10::Device dev = first(gy, "grad_y");
  no_grad(gy);
  const int64_t T = gy.size(0), H = gy.size(1);
  const emu_out_t type = float_type(gy.scalar_type(), "grad_y");
  const int64_t ldy = rows_of(gy, "grad_y", T, H, gy.scalar_type(), dev);
  const at::Tensor kept = given(a[1], "checkpoint", T, 2 * H, at::kFloat8_e4m3fn, dev);
  const at::Tensor kept_scale = given(a[2], "checkpoint_scale", T, 2 * blocks_of(H), at::kFloat, dev);
  On on(dev);
  const at::Tensor out = make({T, 2 * H}, gy.scalar_type(), dev);
  check(emu_swiglu_backward(gy.data_ptr(), ldy, type, T, H, kept.data_ptr(), kept_scale.data_ptr<float>(), out.data_ptr(), on.stream),
        "swiglu_backward");
  return THPVariable_Wrap(out);
}

// One side of a product: codes whose dimensions `row` and `k` are a row and the contraction, the groups' being
// what is left of three.
emu_block_operand_t codes_of(const at::Tensor& t, const char* name, int row, int k, int64_t rows, int64_t K, c10::Device dev) {
  emu_block_operand_t o = {};
  o.format = fp8_type(t.scalar_type(), name);
  if (t.device() != dev) bad(std::string(name) + ": expected on " + dev.str() + ", got " + text(t));
  no_grad(t);
  if (t.size(row) != rows || t.size(k) != K)
    bad(std::string(name) + ": shape mismatch, " + std::to_string(rows) + " by " + std::to_string(K) + " codes expected, got " + text(t));
  o.codes = t.data_ptr();
  o.row_stride = t.stride(row);
  o.k_stride = t.stride(k);
  // a dimension of one has no stride of its own
  if (K <= 1) {
    o.k_stride = 1;
    if (rows <= 1) o.row_stride = 1;
  } else if (rows <= 1) {
    o.row_stride = o.k_stride == 1 ? K : 1;
  }
  if (t.dim() == 3) o.group_stride = t.size(0) <= 1 ? 0 : t.stride(0);
  return o;
}
// its scales: one for each row, or for each 128, by blocks of 128 of K, in any order
void scales_of(emu_block_operand_t& o, const at::Tensor& t, const char* name, int row, int k, int64_t rows, int64_t K, int64_t groups,
               c10::Device dev) {
  no_grad(t);
  const int dims = groups < 0 ? 2 : 3;
  const bool fits = t.dim() == dims && t.scalar_type() == at::kFloat && t.device() == dev && t.size(k) == blocks_of(K) &&
                    (t.size(row) == rows || t.size(row) == blocks_of(rows)) && (dims == 2 || t.size(0) == groups);
  if (!fits)
    bad(std::string(name) + ": fp32 scales expected for " + std::to_string(rows) + " rows, or for each 128 of them, by " +
        std::to_string(blocks_of(K)) + " blocks" + (dims == 3 ? " of " + std::to_string(groups) + " groups" : std::string()) + " on " +
        dev.str() + ", got " + text(t));
  o.scale = static_cast<const float*>(t.data_ptr());
  o.scale_rows = t.size(row) == rows ? 1 : 128;
  o.scale_row_stride = t.stride(row);
  o.scale_k_stride = t.stride(k);
  if (dims == 3) o.scale_group_stride = t.stride(0);
}
at::Tensor workspace_of(PyObject* o, size_t need, c10::Device dev) {
  at::Tensor ws;
  if (o != Py_None) {
    ws = tensor(o, "workspace");
    no_grad(ws);
    if (ws.device() != dev || !ws.is_contiguous()) bad("workspace: a contiguous tensor on " + dev.str() + " expected");
  }
  if (need > 0 && (!ws.defined() || (size_t)ws.nbytes() < need || reinterpret_cast<uintptr_t>(ws.data_ptr()) % 256))
    ws = make({(int64_t)need}, at::kByte, dev);
  return ws;
}
const int32_t* offsets_of(PyObject* o, int64_t groups, c10::Device dev) {
  return static_cast<const int32_t*>(vector_of(tensor(o, "offsets"), "offsets", groups + 1, at::kInt, dev));
}
void same_sides(const at::Tensor& m1, const at::Tensor& m2, int dims) {
  if (m2.dim() != dims) bad("mat2 must be " + std::to_string(dims) + "-D");
  if (m1.size(1) != m2.size(dims - 2)) bad("shape mismatch: " + text(m1) + " @ " + text(m2));
}

// (mat1, mat2, scale_a, scale_b, out_dtype, out, workspace) -> out
PyObject* block_mm(PyObject* const* a) {
  const at::Tensor& m1 = tensor(a[0], "mat1");
  const at::Tensor& m2 = tensor(a[1], "mat2");
  const c10::Device dev = first(m1, "mat1");
  same_sides(m1, m2, 2);
  const int64_t M = m1.size(0), K = m1.size(1), N = m2.size(1);
  emu_block_operand_t oa = codes_of(m1, "mat1", 0, 1, M, K, dev), ob = codes_of(m2, "mat2", 1, 0, N, K, dev);
  scales_of(oa, tensor(a[2], "scale_a"), "scale_a", 0, 1, M, K, -1, dev);
  scales_of(ob, tensor(a[3], "scale_b"), "scale_b", 1, 0, N, K, -1, dev);
  const c10::ScalarType ot = dtype(a[4], "out_dtype");
  const emu_out_t type = out_type(ot);
  On on(dev);
  const at::Tensor out = a[5] == Py_None ? make({M, N}, ot, dev) : given(a[5], "out", M, N, ot, dev);
  const size_t need = emu_block_mm_workspace_bytes(&oa, &ob, M, N, K);
  const at::Tensor ws = workspace_of(a[6], need, dev);
  check(emu_block_scaled_mm(&oa, &ob, M, N, K, out.data_ptr(), type, need ? ws.data_ptr() : nullptr, need, on.stream),
        "block_scaled_mm");
  if (a[5] != Py_None) written(out);
  return a[5] == Py_None ? THPVariable_Wrap(out) : same(a[5]);
}

// (mat1, mat2, offsets, scale_a, scale_b, out_dtype, out, workspace) -> out
PyObject* grouped_mm(PyObject* const* a) {
  const at::Tensor& m1 = tensor(a[0], "mat1");
  const at::Tensor& m2 = tensor(a[1], "mat2");
  const c10::Device dev = first(m1, "mat1");
  same_sides(m1, m2, 3);
  const int64_t T = m1.size(0), K = m1.size(1), E = m2.size(0), N = m2.size(2);
  const int32_t* offsets = offsets_of(a[2], E, dev);
  emu_block_operand_t oa = codes_of(m1, "mat1", 0, 1, T, K, dev), ob = codes_of(m2, "mat2", 2, 1, N, K, dev);
  scales_of(oa, tensor(a[3], "scale_a"), "scale_a", 0, 1, T, K, -1, dev);
  scales_of(ob, tensor(a[4], "scale_b"), "scale_b", 2, 1, N, K, E, dev);
  const c10::ScalarType ot = dtype(a[5], "out_dtype");
  const emu_out_t type = out_type(ot);
  On on(dev);
  const at::Tensor out = a[6] == Py_None ? make({T, N}, ot, dev) : given(a[6], "out", T, N, ot, dev);
  const size_t need = emu_grouped_block_mm_workspace_bytes(&oa, &ob, T, N, K, E);
  const at::Tensor ws = workspace_of(a[7], need, dev);
  check(emu_grouped_block_scaled_mm(&oa, &ob, offsets, E, T, N, K, out.data_ptr(), type, a[6] == Py_None,
                                    need ? ws.data_ptr() : nullptr, need, on.stream), "grouped_block_scaled_mm");
  if (a[6] != Py_None) written(out);
  return a[6] == Py_None ? THPVariable_Wrap(out) : same(a[6]);
}

// the two row-major operands of a weights' gradient: T tokens each
void wgrad_operands(const at::Tensor& g, const at::Tensor& x, emu_block_operand_t& oa, emu_block_operand_t& ob, c10::Device dev) {
  if (x.dim() != 2) bad("x must be 2-D");
  const int64_t T = g.size(0), N = g.size(1), K = x.size(1);
  oa = codes_of(g, "grad", 1, 0, N, T, dev);
  ob = codes_of(x, "x", 1, 0, K, T, dev);
  oa.row_stride = ob.row_stride = 1;
  oa.k_stride = rows_of(g, "grad", T, N, g.scalar_type(), dev);
  ob.k_stride = rows_of(x, "x", T, K, x.scalar_type(), dev);
}
// (grad, x, offsets, scale_grad, scale_x, out_dtype, out, workspace) -> out
PyObject* grouped_wgrad(PyObject* const* a) {
  const at::Tensor& g = tensor(a[0], "grad");
  const at::Tensor& x = tensor(a[1], "x");
  const c10::Device dev = first(g, "grad");
  emu_block_operand_t oa, ob;
  wgrad_operands(g, x, oa, ob, dev);
  const int64_t T = g.size(0), N = g.size(1), K = x.size(1);
  const at::Tensor& off = tensor(a[2], "offsets");
  if (off.dim() != 1 || off.size(0) < 1) bad("offsets must hold the groups' number and one more, got " + text(off));
  const int64_t E = off.size(0) - 1;
  const int32_t* offsets = offsets_of(a[2], E, dev);
  scales_of(oa, tensor(a[3], "scale_grad"), "scale_grad", 1, 0, N, T, -1, dev);
  scales_of(ob, tensor(a[4], "scale_x"), "scale_x", 1, 0, K, T, -1, dev);
  const c10::ScalarType ot = dtype(a[5], "out_dtype");
  const emu_out_t type = out_type(ot);
  On on(dev);
  at::Tensor out;
  if (a[6] == Py_None) {
    out = make({E, N, K}, ot, dev);
  } else {
    out = tensor(a[6], "out");
    no_grad(out);
    if (out.dim() != 3 || out.size(0) != E || out.size(1) != N || out.size(2) != K || out.scalar_type() != ot || !out.is_contiguous() ||
        out.device() != dev)
      bad("out must be a contiguous " + text(ot) + " (" + std::to_string(E) + ", " + std::to_string(N) + ", " + std::to_string(K) +
          ") on " + dev.str() + ", got " + text(out));
  }
  const size_t need = emu_grouped_block_wgrad_workspace_bytes(&oa, &ob, T, N, K);
  const at::Tensor ws = workspace_of(a[7], need, dev);
  check(emu_grouped_block_scaled_wgrad(&oa, &ob, offsets, E, T, N, K, out.data_ptr(), type, need ? ws.data_ptr() : nullptr, need,
                                       on.stream), "grouped_block_scaled_wgrad");
  if (a[6] != Py_None) written(out);
  return a[6] == Py_None ? THPVariable_Wrap(out) : same(a[6]);
}

// (mat1, mat2) -> bytes; mat2 of three dimensions: by group
PyObject* block_mm_bytes(PyObject* const* a) {
  const at::Tensor& m1 = tensor(a[0], "mat1");
  const at::Tensor& m2 = tensor(a[1], "mat2");
  const c10::Device dev = first(m1, "mat1");
  const int dims = m2.dim() == 3 ? 3 : 2;
  same_sides(m1, m2, dims);
  const int64_t M = m1.size(0), K = m1.size(1), N = m2.size(dims - 1);
  const emu_block_operand_t oa = codes_of(m1, "mat1", 0, 1, M, K, dev), ob = codes_of(m2, "mat2", dims - 1, dims - 2, N, K, dev);
  return PyLong_FromSize_t(dims == 3 ? emu_grouped_block_mm_workspace_bytes(&oa, &ob, M, N, K, m2.size(0))
                                     : emu_block_mm_workspace_bytes(&oa, &ob, M, N, K));
}
// (grad, x) -> bytes
PyObject* block_wgrad_bytes(PyObject* const* a) {
  const at::Tensor& g = tensor(a[0], "grad");
  const at::Tensor& x = tensor(a[1], "x");
  emu_block_operand_t oa, ob;
  wgrad_operands(g, x, oa, ob, first(g, "grad"));
  return PyLong_FromSize_t(emu_grouped_block_wgrad_workspace_bytes(&oa, &ob, g.size(0), g.size(1), x.size(1)));
}
