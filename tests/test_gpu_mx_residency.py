"""What a product's blocks leave of an SM to others."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k", [(1, 512, 8192), (16, 4096, 4096), (64, 8192, 4096), (2048, 1280, 512), (1, 11008, 4096)])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_blocks_that_wait_for_each_other_have_their_sms_alone(fmt, m, n, k):
    """Clusters take all of the shared memory, so that no block of another kernel is beside one
    with the tensor memory that its neighbour waits for."""
    driver = pytest.importorskip("cuda.bindings.driver")
    from lossless_float_weight_b200 import mx
    a, b = (mx.quantize(torch.ones(r, k, device="cuda"), fmt) for r in (m, n))
    out = mx.matmul(a, b)
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        mx.matmul(a, b, out=out)
    graph = driver.CUgraph(g.raw_cuda_graph())
    err, nodes, count = driver.cuGraphGetNodes(graph, 4)
    assert err == driver.CUresult.CUDA_SUCCESS and count == 1
    err, params = driver.cuGraphKernelNodeGetParams(nodes[0])
    assert err == driver.CUresult.CUDA_SUCCESS
    err, cluster = driver.cuGraphKernelNodeGetAttribute(nodes[0], driver.CUkernelNodeAttrID.CU_LAUNCH_ATTRIBUTE_CLUSTER_DIMENSION)
    waits = err == driver.CUresult.CUDA_SUCCESS and cluster.clusterDim.x > 1
    assert waits == (n != 11008)
    if waits:
        assert params.sharedMemBytes == 227 * 1024
