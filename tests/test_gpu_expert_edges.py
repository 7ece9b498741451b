"""Routing, gradients and products at the edges of their ranges, on the GPU against float64."""
import pytest
import torch

import scaled_oracle as O
from tensor_gemm_reduction_amd import tpfuse as tp

pytestmark = pytest.mark.gpu
