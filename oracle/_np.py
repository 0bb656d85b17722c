"""Tensors to numpy for the oracle.  TEST INFRASTRUCTURE ONLY."""
import numpy as np
import torch


def to_np(x):
    """float64 (floating tensors), the integer type, or the array as given."""
    if isinstance(x, torch.Tensor):
        return (x.detach().double() if x.is_floating_point() else x.detach()).cpu().numpy()
    return np.asarray(x)
