"""Codes and scale bytes that stand by rows, brought into the form of the 4-bit operators as mx4.py says."""
import numpy as np
import pytest
import torch

import mx4_reference as ref
import weight_quantization_codec_amd as q


@pytest.mark.parametrize("rows,d", [(1, 1), (3, 31), (2, 64), (5, 257), (4, 512), (7, 1003)])
def test_bytes_by_rows(rows, d):
    want = ref.quantize(np.random.default_rng(rows + d).standard_normal((rows, d)).astype(np.float32))
    codes = torch.from_numpy(want[0][:, :(d + 1) // 2].copy())
    scales = torch.from_numpy(want[1].transpose(1, 0, 2).reshape(rows, -1)[:, :(d + 31) // 32].copy())
    doc = q.mx4.__doc__
    steps = [line.strip() for line in doc.splitlines() if line.startswith("    ")]
    assert len(steps) == 3
    names = dict(torch=torch, codes=codes, scales=scales, rows=rows, d=d, mx4_stride=q.mx4_stride, mx4_groups=q.mx4_groups)
    exec("\n".join(steps), names)
    assert np.array_equal(names["codes"].numpy(), want[0]) and np.array_equal(names["scales"].numpy(), want[1])
    assert names["codes"].is_contiguous() and names["scales"].is_contiguous()
